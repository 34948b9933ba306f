"""What the quantised cache's and the drafted trees' operators are timed on, with their plain forms.

The target's forward pass over a paged cache whose 8-bit entries carry a scale for
every token and kv head, taken as the token is written; and over drafts that form a
tree, several continuations of one sequence judged in one pass.

  append   the new tokens' keys and values, quantised, into their pages (dspark.cache_append, cache "f8t")
  attend   attention of each request's new tokens over such pages (dspark.cache_attend, cache "f8t")
  mask     a drafted tree's ancestors and depths from its parents (dspark.tree_mask)
  tree     attention of a tree's nodes over the cache and their ancestors (dspark.tree_attend)
  keep     the accepted nodes' keys and values moved to the front of the tree (dspark.tree_keep)

``own`` false: elementary torch operations in 32 bits.  ``own`` true: the library's
calls.  ``exact``: the same outputs in 64 bits, from the definitions.

Cache layout (both forms): keys [layers][pages][Hkv][page][D], values
[layers][pages][Hkv][page/8][D][8] (groups of 8 tokens, token fastest); with a scale a
token ("f8t"), each page and head is page * D bytes in that order, then page fp32 scales.
"""
import math

import numpy as np
import torch

own = False

_DATA = {"bf16": torch.bfloat16, "f32": torch.float32, "f8": torch.bfloat16, "f8t": torch.bfloat16}
_STORE = {"bf16": torch.bfloat16, "f32": torch.float32, "f8": torch.float8_e4m3fn, "f8t": torch.float8_e4m3fn}
_BYTES = {"bf16": 2, "f32": 4, "f8": 1, "f8t": 1}
_E4M3 = 448.0


# ------------------------------------------------------------------ cases
def listed():
    def rows(name, op, B, T, S, Hq, Hkv, D, page, dtype, window=0):
        return dict(name=name, op=op, B=B, T=T, S=S, Hq=Hq, Hkv=Hkv, D=D, page=page, dtype=dtype, window=window)

    def append(name, B, T, S, Hkv, D, page):
        return dict(name=name, op="append", B=B, T=T, S=S, Hkv=Hkv, D=D, page=page, dtype="f8t")

    return [
        # new tokens of a verification cycle at the headline concurrency (K + 1 = 17), each quantised by its own scale
        append("append verify", 256, 17, 1024, 8, 128, 16),
        # prompt chunks
        append("append prompt chunk", 4, 2048, 8192, 8, 128, 64),
        # plain decoding, one token for each of 256 concurrent requests, ragged contexts
        rows("attend token batch", "attend", 256, 1, 4096, 32, 8, 128, 64, "f8t"),
        # the verification forward of the headline workload, ragged
        rows("attend verify batch", "attend", 256, 17, 2048, 32, 8, 128, 16, "f8t"),
        # prompt chunks of four requests over their earlier context
        rows("attend prompt chunk", "attend", 4, 2048, 8192, 32, 8, 128, 32, "f8t"),
        # one request of the smallest configuration (hidden size 128 = 2 heads x 64, fp32) with a tree of 8: latency
        rows("tree tiny", "tree", 1, 8, 500, 2, 2, 64, 16, "f32"),
        # trees of up to 64 drafts for 64 requests
        rows("tree batch", "tree", 64, 64, 4096, 32, 8, 128, 64, "bf16"),
        # few requests with long contexts and large trees, quantised cache
        rows("tree large", "tree", 8, 256, 32768, 32, 4, 128, 256, "f8t"),
        # one small tree
        dict(name="mask small", op="mask", B=1, T=16, window=0),
        # the trees of a batch, for a layer with a sliding window
        dict(name="mask batch", op="mask", B=256, T=64, window=4),
        # the accepted path of one tree, all layers of the smallest configuration's kind
        dict(name="keep small", op="keep", B=1, T=16, S=500, path=5, layers=2, Hkv=2, D=64, page=16, dtype="f32"),
        # the accepted paths of a batch in all layers of a part of the target
        dict(name="keep batch", op="keep", B=256, T=32, S=512, path=8, layers=4, Hkv=8, D=128, page=16, dtype="bf16"),
    ]


def _logint(rng, lo, hi):
    return int(min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "mask", "tree", "tree", "keep"])
    page = rng.choice([16, 32, 64, 128, 256])
    D = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    dtype = rng.choice(["bf16", "bf16", "f8", "f8t", "f32"])
    if op == "mask":
        return dict(op=op, B=_logint(rng, 1, 256), T=_logint(rng, 1, 256), window=rng.choice([0, 0, _logint(rng, 1, 16)]))
    if op == "append":
        T = rng.choice([1, _logint(rng, 1, 33), _logint(rng, 64, 2048)])
        B = _logint(rng, 1, 256 if T <= 33 else 4)
        S = _logint(rng, 1, max(1, min(8192, (1 << 28) // (B * Hkv * D))))
        return dict(op=op, B=B, T=T, S=S, Hkv=Hkv, D=D, page=page, dtype="f8t")
    if op == "keep":
        B, layers = _logint(rng, 1, 256), rng.choice([1, 2, 4])
        S = _logint(rng, 1, max(1, min(4096, (1 << 27) // (B * Hkv * D * layers))))
        return dict(op=op, B=B, T=_logint(rng, 1, 64), S=S, path=_logint(rng, 1, 12), layers=layers, Hkv=Hkv, D=D, page=page,
                    dtype=dtype)
    if op == "attend":
        T, dtype = rng.choice([1, _logint(rng, 1, 33), _logint(rng, 1, 33), _logint(rng, 64, 2048)]), "f8t"
    else:
        T = rng.choice([_logint(rng, 1, 33), _logint(rng, 8, 256)])
    Hq = Hkv * rng.choice([1, 2, 4, 5, 8])
    B = _logint(rng, 1, 256 if T <= 33 else 16 if T <= 256 else 4)
    # at most half a GiB of elements in a pool and 4 GiB of scores in the plain form
    most = min((1 << 29) // (B * Hkv * D), (1 << 30) // (B * T * Hq), 200000)
    return dict(op=op, B=B, T=T, S=_logint(rng, 1, max(1, most)), Hq=Hq, Hkv=Hkv, D=D, page=page, dtype=dtype,
                window=rng.choice([0, 0, 0, _logint(rng, 1, 4096)]))


def _ceil(a, b):
    return -(-a // b)


def _rows_of(c):
    """New tokens of the requests, before the seed's order: ragged, one of five without any where there are several."""
    i = np.arange(c["B"])
    n = np.full(c["B"], c["T"]) if (c["op"] in ("append", "attend") and c["T"] > 33) or c["B"] == 1 else 1 + (i * 5) % c["T"]
    if c["B"] >= 5 and c["T"] > 1:
        n[i % 5 == 3] = 0
        n[-1] = c["T"]
    return n


def _lengths(c):
    n = _rows_of(c)
    s = np.maximum(n, np.round(c["S"] * (0.1 + 0.9 * (np.arange(c["B"]) + 1) / c["B"])).astype(np.int64))
    return n, s


def _path_of(c, n):
    """Accepted nodes of the requests: up to `path` of the nodes that there are."""
    return np.minimum(n, 1 + np.arange(c["B"]) % c["path"])


def work(case):
    c = case
    if c["op"] == "mask":
        rows, words = int(_rows_of(c).sum()), _ceil(c["T"], 32)
        return {"bytes": 4 * rows * (2 + words) + 8 * c["B"], "flops": 0}
    n, s = _lengths(c)
    # bytes of a token and head: the entries, and a scale each of the key and the value
    data, held = 4 if c["dtype"] == "f32" else 2, 2 * (c["D"] * _BYTES[c["dtype"]] + (4 if c["dtype"] == "f8t" else 0))
    rows = int(n.sum())
    if c["op"] == "append":
        return {"bytes": rows * c["Hkv"] * (2 * c["D"] * data + held), "flops": 0}
    if c["op"] == "keep":
        return {"bytes": int(_path_of(c, n).sum()) * c["layers"] * c["Hkv"] * 2 * held + 16 * c["B"], "flops": 0}
    first = np.maximum(0, s - n - c["window"] + 1) if c["window"] else np.zeros_like(s)
    keys = int(np.where(n > 0, s - first, 0).sum())
    pairs = 0
    for nb, sb in zip(n, s):
        pos = sb - nb + (np.arange(nb) if c["op"] == "attend" else np.zeros(nb, int))  # (a tree's node: its context, itself)
        lo = np.maximum(0, pos - c["window"] + 1) if c["window"] else 0
        pairs += int((pos + 1 - lo).sum())
    byts = keys * c["Hkv"] * held + rows * c["Hq"] * (2 * c["D"] * data + 4)
    return {"bytes": byts + (4 * rows * _ceil(c["T"], 32) if c["op"] == "tree" else 0), "flops": 4 * pairs * c["Hq"] * c["D"]}


# ------------------------------------------------------------------ inputs
def _views(c, pool, values):
    """Entries and scales (or None) of a pool, as views."""
    if c["dtype"] != "f8t":
        return pool, None
    layers, pages, Hkv, _ = pool.shape
    page, D = c["page"], c["D"]
    shape = (page // 8, D, 8) if values else (page, D)
    return (pool[..., :page * D].view(torch.float8_e4m3fn).unflatten(3, shape),
            pool.view(torch.float32)[..., page * D // 4:])


def _pool(c, n_pages, layers, values, gen):
    page, D, Hkv = c["page"], c["D"], c["Hkv"]
    shape = (layers, n_pages, Hkv, page // 8, D, 8) if values else (layers, n_pages, Hkv, page, D)
    if c["dtype"] in ("bf16", "f32"):
        return torch.randn(shape, dtype=_STORE[c["dtype"]], device="cuda", generator=gen)
    t = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
    std = 40.0 if c["dtype"] == "f8" else 120.0
    for a in t.view(-1).split(1 << 28):
        a.copy_(torch.randn(a.shape, dtype=torch.bfloat16, device="cuda", generator=gen).mul_(std).clamp_(-448, 448))
    if c["dtype"] == "f8":
        return t
    pool = torch.empty(layers, n_pages, Hkv, page * (D + 4), dtype=torch.uint8, device="cuda")
    entries, scales = _views(c, pool, values)
    entries.view(torch.uint8).copy_(t.view(torch.uint8))
    # tokens of rows of about unit size, some of them many times larger
    scales.copy_(torch.randn(scales.shape, device="cuda", generator=gen).mul_(0.5).exp_().mul_(0.008))
    return pool


def _i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def _trees(rng, n):
    """Parents of the requests' nodes: node 0 is the anchor (-1: the context alone), the others hang from earlier ones."""
    rows, start = int(n.sum()), np.cumsum(n) - n
    i = np.arange(rows) - np.repeat(start, n)
    at = (i // 3 + rng.random(rows) * (i - i // 3)).astype(np.int64)
    return np.where(i == 0, -1, np.minimum(at, i - 1)), i, start


def _ancestors(parent, i, start, n, T, window):
    """Ancestor bits (a node's own among them) and depths, node by node."""
    mask = np.zeros((len(parent), T), bool)
    depth = np.zeros(len(parent), np.int64)
    first = np.repeat(start, n)
    for k in range(int(n.max()) if len(n) else 0):
        r = np.flatnonzero(i == k)
        up = parent[r]
        has = up >= 0
        mask[r[has]] = mask[first[r[has]] + up[has]]
        depth[r[has]] = depth[first[r[has]] + up[has]] + 1
        mask[r, k] = True
    if window:
        for b, m in enumerate(n):
            d = depth[start[b]:start[b] + m]
            mask[start[b]:start[b] + m, :m] &= d[:, None] - d[None, :] < window
    return mask, depth


def _words(mask):
    """Bits [rows][T] as int32 words [rows][ceil(T / 32)]."""
    rows, T = mask.shape
    full = np.zeros((rows, _ceil(T, 32) * 32), np.uint8)
    full[:, :T] = mask
    return np.packbits(full, 1, bitorder="little").view("<i4").astype(np.int64).reshape(rows, -1)


def prepare(case, seed):
    c = case
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    randn = lambda *shape: torch.randn(shape, device="cuda", generator=gen)  # noqa: E731
    st = dict(c=c)
    order = rng.permutation(c["B"])
    if c["op"] == "mask":
        n = _rows_of(c)[order]
        parent, _, start = _trees(rng, n)
        st["parent"], st["n_new"], st["row_start"] = _i32(parent), _i32(n), _i32(start)
        st["mask"] = torch.empty(len(parent), _ceil(c["T"], 32), dtype=torch.int32, device="cuda")
        st["depth"] = torch.empty(len(parent), dtype=torch.int32, device="cuda")
        return st
    n, s = (x[order] for x in _lengths(c))
    width = _ceil(int(s.max()), c["page"])
    held = _ceil(s, c["page"])
    n_pages = int(held.sum()) + 3
    ids = rng.permutation(n_pages)
    table = np.full((c["B"], width), -1, np.int64)
    for b, at in enumerate(np.cumsum(held) - held):
        table[b, :held[b]] = ids[at:at + held[b]]
    layers = c.get("layers", 1)
    st["k_pool"], st["v_pool"] = (_pool(c, n_pages, layers, x, gen) for x in (False, True))
    st["k_scale"], st["v_scale"] = (randn(c["Hkv"]).abs_().mul_(0.01).add_(0.02) if c["dtype"] == "f8" else None
                                    for _ in range(2))
    st["n_new"], st["row_start"] = _i32(n), _i32(np.cumsum(n) - n)
    st["length"], st["table"] = _i32(s), _i32(table)
    rows, data = int(n.sum()), _DATA[c["dtype"]]
    if c["op"] == "append":
        kv = randn(rows, 2 * c["Hkv"], c["D"]).mul_(randn(rows, 1, 1).exp_()).to(data)  # one projection's output
        st["k"], st["v"] = kv[:, :c["Hkv"]], kv[:, c["Hkv"]:]
    elif c["op"] == "keep":
        parent, _, start = _trees(rng, n)
        want = _path_of(c, n)
        path, m = np.full((c["B"], c["path"]), -1, np.int64), np.zeros(c["B"], np.int64)
        for b in range(c["B"]):  # the root, then from a deep node up as far as the path is long
            if n[b] == 0:
                continue
            up, node = [], int(rng.integers(n[b] // 2, n[b]))
            while node >= 0:
                up.append(node)
                node = int(parent[start[b] + node])
            got = up[::-1][:want[b]]
            path[b, :len(got)], m[b] = got, len(got)
        st["path"], st["n_keep"] = _i32(path), _i32(m)
        st["length_out"] = torch.empty(c["B"], dtype=torch.int32, device="cuda")
    else:
        # queries a little wider than unit normal: softmax maps with some peaks
        st["q"] = randn(rows, c["Hq"], c["D"]).mul_(1.5).to(data)
        st["out"] = torch.empty(rows, c["Hq"], c["D"], dtype=data, device="cuda")
        st["lse"] = torch.empty(rows, c["Hq"], dtype=torch.float32, device="cuda")
        if c["op"] == "tree":
            parent, i, start = _trees(rng, n)
            mask, depth = _ancestors(parent, i, start, n, c["T"], c["window"])
            st["mask"], st["depth"] = _i32(_words(mask)), _i32(depth)
    if own:
        from draft_sampling_verification_markov_amd import dspark
        C = dspark.Cache.make(c["B"], n_pages, c["page"], width, layers, c.get("Hq", c["Hkv"]), c["Hkv"], c["D"],
                              q="f32" if c["dtype"] == "f32" else "bf16", cache=c["dtype"])
        st["C"] = C
        st["ws"] = torch.empty(dspark.cache_workspace_bytes(C, c["T"]), dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------------ plain forms
def _bytes_of(x):
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x


def _dense(st, which, pages):
    """The only layer's keys or values of these pages as [B][Hkv][tokens][D] in 32 bits."""
    c, values = st["c"], which == "v"
    entries, scales = _views(c, st[which + "_pool"], values)
    x = _bytes_of(entries)[0][pages]  # [B][P][Hkv][...]
    x = (x.view(torch.float8_e4m3fn) if _BYTES[c["dtype"]] == 1 else x).float()
    if values:  # [B][P][Hkv][page/8][D][8]
        x = x.transpose(4, 5).flatten(3, 4)
    if scales is not None:
        x = x * scales[0][pages][..., None]
    x = x.transpose(1, 2).flatten(2, 3)
    return x * st[which + "_scale"][:, None, None] if c["dtype"] == "f8" else x


def _attend(st):
    c = st["c"]
    B, T, Hkv, G, D = c["B"], c["T"], c["Hkv"], c["Hq"] // c["Hkv"], c["D"]
    dev = st["q"].device
    n, s, start = st["n_new"].long(), st["length"].long(), st["row_start"].long()
    t = torch.arange(T, device=dev)
    at = (start[:, None] + t).clamp(max=st["q"].shape[0] - 1)
    q = st["q"].float()[at]  # [B][T][Hq][D]
    q = q.view(B, T, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, D)
    page, width = c["page"], st["table"].shape[1]
    slot = torch.arange(width, device=dev).expand(B, -1)
    if c["window"]:  # no key before the first new token's window is needed
        slot = ((s - n - c["window"] + 1).clamp(min=0) // page)[:, None] + slot[:, :_ceil(c["window"] + T - 1, page) + 1]
    pages = st["table"].gather(1, slot.clamp(max=width - 1)).clamp(min=0).long()  # (a slot that is not held: page 0)
    k, v = _dense(st, "k", pages), _dense(st, "v", pages)
    j = (slot[..., None] * page + torch.arange(page, device=dev)).flatten(1)[:, None]  # [B][1][keys]
    base = (s - n)[:, None]
    seen = (j < s[:, None, None]).expand(B, T, -1)
    if c["op"] == "tree":
        bits = (st["mask"][at][..., None] >> torch.arange(32, device=dev) & 1).flatten(2) > 0  # [B][T][words * 32]
        node = j - base[..., None]
        among = bits.gather(2, node.clamp(0, bits.shape[2] - 1).expand(B, T, -1))
        seen = seen & ((node < 0) | among)
        pos = base + st["depth"].long()[at]
        if c["window"]:
            seen = seen & ((node >= 0) | (j > pos[..., None] - c["window"]))
    else:
        pos = base + t  # [B][T]
        seen = seen & (j <= pos[..., None])
        if c["window"]:
            seen = seen & (j > pos[..., None] - c["window"])
    seen = seen[:, None, :, None, :]
    score = torch.matmul(q, k.transpose(2, 3)).mul_(D ** -0.5).view(B, Hkv, T, G, -1)
    score = score.masked_fill_(~seen, -math.inf)
    top = score.amax(-1, keepdim=True).clamp_(min=torch.finfo(torch.float32).min)
    p = score.sub_(top).exp_()
    total = p.sum(-1)
    o = torch.matmul(p.view(B, Hkv, T * G, -1), v.masked_fill_((j >= s[:, None, None])[..., None], 0.0))
    o = o.view(B, Hkv, T, G, D) / total.clamp(min=1e-37)[..., None]
    lse = top[..., 0] + total.log()
    row = torch.arange(st["q"].shape[0], device=dev)
    end = torch.cumsum(n, 0)
    b = torch.searchsorted(end, row, right=True)
    i = row - start[b]
    o = o.permute(0, 2, 1, 3, 4)[b, i].reshape(-1, c["Hq"], D)
    return [o.to(st["q"].dtype), lse.permute(0, 2, 1, 3)[b, i].reshape(-1, c["Hq"])]


def _quantise(x):
    """Entries (as bytes) and the scale of each row: its largest size goes to 448, the largest e4m3 value."""
    x = x.float()
    top = x.abs().amax(-1)
    scale = torch.where(top > 0, (top / _E4M3).clamp(min=2.0 ** -126), 1.0)
    return (x / scale[..., None]).clamp(-_E4M3, _E4M3).to(torch.float8_e4m3fn).view(torch.uint8), scale


def _append(st):
    c = st["c"]
    n, s, start = st["n_new"].long(), st["length"].long(), st["row_start"].long()
    row = torch.arange(st["k"].shape[0], device="cuda")
    b = torch.searchsorted(torch.cumsum(n, 0), row, right=True)
    pos = s[b] - n[b] + row - start[b]
    page = st["table"].long()[b, pos // c["page"]]
    off = pos % c["page"]
    (k, ks), (v, vs) = _views(c, st["k_pool"], False), _views(c, st["v_pool"], True)
    (kq, kt), (vq, vt) = _quantise(st["k"]), _quantise(st["v"])
    k[0].view(torch.uint8)[page, :, off] = kq
    v[0].view(torch.uint8)[page, :, off // 8, :, off % 8] = vq
    ks[0][page, :, off] = kt
    vs[0][page, :, off] = vt
    return [k, ks, v, vs]


def _mask(st):
    c = st["c"]
    B, T = c["B"], c["T"]
    n, start = st["n_new"].long(), st["row_start"].long()
    t = torch.arange(T, device="cuda")
    rows = (start[:, None] + t).clamp(max=st["parent"].numel() - 1)
    parent = torch.where(t < n[:, None], st["parent"].long()[rows], -1)
    up = (parent[..., None] == t).float() + torch.eye(T, device="cuda")  # a node, and its parent
    for _ in range(max(1, (T - 1).bit_length())):
        up = (torch.matmul(up, up) > 0).float()
    depth = up.sum(-1).long() - 1
    seen = up > 0
    if c["window"]:
        seen = seen & (depth[:, :, None] - depth[:, None, :] < c["window"])
    words = torch.zeros(B, T, _ceil(T, 32) * 32, dtype=torch.int64, device="cuda")
    words[..., :T] = seen
    words = (words.view(B, T, -1, 32) << torch.arange(32, device="cuda")).sum(-1)
    words = torch.where(words >= 1 << 31, words - (1 << 32), words).int()
    row = torch.arange(st["parent"].numel(), device="cuda")
    b = torch.searchsorted(torch.cumsum(n, 0), row, right=True)
    i = row - start[b]
    return [words[b, i], depth[b, i].int()]


def _keep(st):
    c = st["c"]
    n, s, m, path = (st[x].long() for x in ("n_new", "length", "n_keep", "path"))
    i = torch.arange(path.shape[1], device="cuda")
    b, i = torch.nonzero(i < m[:, None], as_tuple=True)
    base, table = s - n, st["table"].long()
    src, dst = base[b] + path[b, i], base[b] + i
    ps, pd = table[b, src // c["page"]], table[b, dst // c["page"]]
    so, do = src % c["page"], dst % c["page"]
    out = []
    for which in "kv":
        x, scales = _views(c, st[which + "_pool"], which == "v")
        raw = _bytes_of(x)
        if which == "k":
            raw[:, pd, :, do] = raw[:, ps, :, so]
        else:
            raw[:, pd, :, do // 8, :, do % 8] = raw[:, ps, :, so // 8, :, so % 8]
        out.append(x)
        if scales is not None:
            scales[:, pd, :, do] = scales[:, ps, :, so]
            out.append(scales)
    st["length_out"].copy_(base + m)
    return out + [st["length_out"]]


def run(state):
    st, c = state, state["c"]
    if not own:
        return {"append": _append, "attend": _attend, "mask": _mask, "tree": _attend, "keep": _keep}[c["op"]](st)
    from draft_sampling_verification_markov_amd import dspark
    if c["op"] == "mask":
        dspark.tree_mask(st["parent"], st["n_new"], st["row_start"], c["T"], st["mask"], st["depth"], window=c["window"])
        return [st["mask"], st["depth"]]
    C = st["C"]
    if c["op"] == "append":
        dspark.cache_append(C, 0, st["k"], st["v"], st["n_new"], st["row_start"], c["T"], st["length"], st["table"],
                            None, None, st["k_pool"], st["v_pool"])
        return [*_views(c, st["k_pool"], False), *_views(c, st["v_pool"], True)]
    if c["op"] == "attend":
        dspark.cache_attend(C, 0, st["q"], st["n_new"], st["row_start"], c["T"], st["length"], st["table"], st["k_pool"],
                            st["v_pool"], None, None, st["out"], st["lse"], st["ws"], window=c["window"])
        return [st["out"], st["lse"]]
    if c["op"] == "tree":
        dspark.tree_attend(C, 0, st["q"], st["n_new"], st["row_start"], c["T"], st["mask"], st["depth"], st["length"],
                           st["table"], st["k_pool"], st["v_pool"], st["k_scale"], st["v_scale"], st["out"], st["lse"],
                           st["ws"], window=c["window"])
        return [st["out"], st["lse"]]
    dspark.tree_keep(C, st["path"], st["n_keep"], st["n_new"], c["T"], st["length"], st["table"], st["length_out"],
                     st["k_pool"], st["v_pool"])
    pools = [x for w in "kv" for x in _views(c, st[w + "_pool"], w == "v") if x is not None]
    return pools + [st["length_out"]]


# ------------------------------------------------------------------ 64 bits, from the definitions
def _exact_rows(st, which, h, pages, s):
    """Head h's first s keys or values of a sequence in 64 bits, [s][D]."""
    c = st["c"]
    x, scales = _views(c, st[which + "_pool"], which == "v")
    x = _bytes_of(x)[0][pages, h]
    x = (x.view(torch.float8_e4m3fn) if _BYTES[c["dtype"]] == 1 else x).double()
    if which == "v":
        x = x.permute(0, 1, 3, 2)
    x = x.reshape(-1, c["D"])[:s]
    if scales is not None:
        x = x * scales[0][pages, h].double().reshape(-1)[:s, None]
    return x * st[which + "_scale"][h].double() if c["dtype"] == "f8" else x


def _exact_attend(st):
    c = st["c"]
    G, page = c["Hq"] // c["Hkv"], c["page"]
    out, lse = st["q"].double(), torch.empty(st["q"].shape[:2], dtype=torch.float64, device="cuda")
    for n, s, r, pages in zip(*(st[x].tolist() for x in ("n_new", "length", "row_start", "table"))):
        if n == 0:
            continue
        pages = torch.tensor(pages[:_ceil(s, page)], device="cuda", dtype=torch.long)
        j, i = torch.arange(s, device="cuda"), torch.arange(n, device="cuda")[:, None]
        base = s - n
        if c["op"] == "tree":
            hidden = torch.zeros(n, s, dtype=torch.bool, device="cuda")
            words = st["mask"][r:r + n].cpu().numpy().astype("<i4").view(np.uint8)
            among = np.unpackbits(words.reshape(n, -1), axis=1, bitorder="little")[:, :n] != 0
            hidden[:, base:] = ~torch.from_numpy(among).cuda()
            if c["window"]:
                hidden[:, :base] |= j[:base] + c["window"] <= base + st["depth"][r:r + n, None]
        else:
            hidden = j > base + i
            if c["window"]:
                hidden |= j + c["window"] <= base + i
        for h in range(c["Hkv"]):
            k, v = (_exact_rows(st, w, h, pages, s) for w in "kv")
            x = st["q"][r:r + n, h * G:(h + 1) * G].double().reshape(n * G, -1) @ k.t().contiguous() / math.sqrt(c["D"])
            x = x.view(n, G, s).masked_fill(hidden[:, None], -math.inf)
            z = torch.logsumexp(x, -1)
            p = torch.where(hidden[:, None], 0.0, torch.exp(x - z.nan_to_num(neginf=0.0)[..., None]))
            out[r:r + n, h * G:(h + 1) * G] = (p.view(n * G, s) @ v).view(n, G, -1)
            lse[r:r + n, h * G:(h + 1) * G] = z
    return [out, lse]


def _exact_append(st):
    c = st["c"]
    (k, ks), (v, vs) = _views(c, st["k_pool"], False), _views(c, st["v_pool"], True)
    k, ks, v, vs = k.double(), ks.double(), v.double(), vs.double()
    page, off, row = [], [], []
    for n, s, r, pages in zip(*(st[x].tolist() for x in ("n_new", "length", "row_start", "table"))):
        for i in range(n):
            page.append(pages[(s - n + i) // c["page"]])
            off.append((s - n + i) % c["page"])
            row.append(r + i)
    page, off, row = (torch.tensor(x, device="cuda", dtype=torch.long) for x in (page, off, row))
    for x, scales, new, values in ((k, ks, st["k"], False), (v, vs, st["v"], True)):
        new = new.double()[row]
        scale = new.abs().amax(-1) / _E4M3
        scale[scale == 0] = 1.0
        scales[0][page, :, off] = scale
        if values:
            x[0].permute(0, 1, 2, 4, 3)[page, :, off // 8, off % 8] = new / scale[..., None]
        else:
            x[0][page, :, off] = new / scale[..., None]
    return [k, ks, v, vs]


def _exact_mask(st):
    c = st["c"]
    parent, n, start = (st[x].tolist() for x in ("parent", "n_new", "row_start"))
    words, depth = np.zeros((len(parent), _ceil(c["T"], 32)), np.uint32), np.zeros(len(parent), np.int64)
    for m, r in zip(n, start):
        for i in range(m):
            chain = [i]
            while parent[r + chain[-1]] >= 0:
                chain.append(parent[r + chain[-1]])
            depth[r + i] = len(chain) - 1
            for a in chain[:c["window"]] if c["window"] else chain:
                words[r + i, a // 32] |= np.uint32(1 << a % 32)
    return [_i32(words.view(np.int32)), _i32(depth)]


def _exact_keep(st):
    c = st["c"]
    out = []
    for which in "kv":
        x, scales = _views(c, st[which + "_pool"], which == "v")
        out += [y.double() for y in (x, scales) if y is not None]
    new_len = []
    for n, s, m, path, pages in zip(*(st[x].tolist() for x in ("n_new", "length", "n_keep", "path", "table"))):
        base = s - n
        new_len.append(base + m)
        for i in range(m):  # (a node's place is never one that a later node comes from)
            a, b = base + path[i], base + i
            pa, pb, oa, ob = pages[a // c["page"]], pages[b // c["page"]], a % c["page"], b % c["page"]
            for y in out:
                if y.dim() == 6:
                    y[:, pb, :, ob // 8, :, ob % 8] = y[:, pa, :, oa // 8, :, oa % 8]
                else:
                    y[:, pb, :, ob] = y[:, pa, :, oa]
    return out + [_i32(new_len)]


def exact(case, seed):
    st = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "mask": _exact_mask, "tree": _exact_attend,
            "keep": _exact_keep}[case["op"]](st)
