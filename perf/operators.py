"""Measured cases of the serving-cache and sliding-window operators.

Three operators, used together when a long-context model trains with windowed layers
and then serves from a quantised cache:

  cache   rows of K and V written into a cache (microscaled 8- or 4-bit floats), and
          read back as the values they stand for: cache_write, cache_read
  tree    attention of drafted tokens (a tree, a chain, or one token) over that cache,
          with an optional sliding window and sinks: tree_attention
  window  causal attention in which token t sees the last `window` tokens and the
          first `sinks` tokens, and its gradients: window_attention,
          window_attention_backward

Every operator has its plain form here (elementary torch operations in 32 bits), its
definition in 64 bits (`exact`), and the library calls (`own`).

Microscaled formats: along the head dimension, every block of 32 values shares one
power of two 2^k (stored as the byte k + 127; 255 marks a block with a value that is not
finite), k being the smallest integer with max|x| <= M 2^k. The values are kept as
x 2^-k rounded to nearest even: mxfp8 in e4m3 (M = 448), mxfp4 in e2m1 (M = 6; element
2i in the low half of byte i).
"""
import math

import torch

own = False

_E4M3_MAX_F = 0.875  # 448 = 0.875 * 2^9
_E2M1_MAX_F = 0.75   # 6   = 0.75  * 2^3
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # one new token for each of 64 running sequences, appended to its 8-bit cache
        dict(name="append_fp8", kind="cache", op="write", fmt="mxfp8", B=64, Hkv=8, D=128, T=1, cap=4096, dtype="bf16",
             ragged=False, fused=True),
        # a long prompt's chunk written to a 4-bit cache straight from a fused K/V projection
        dict(name="prefill_fp4", kind="cache", op="write", fmt="mxfp4", B=1, Hkv=8, D=128, T=30011, cap=65536,
             dtype="bf16", ragged=False, fused=True),
        # a prefix read back in bf16 to be attended by the next prompt chunk
        dict(name="read_fp8", kind="cache", op="read", fmt="mxfp8", B=2, Hkv=8, D=128, T=65536, cap=70000, dtype="bf16",
             ragged=False, fused=False),
        # a padded batch of prefixes read back in fp32
        dict(name="read_fp4_ragged", kind="cache", op="read", fmt="mxfp4", B=5, Hkv=4, D=64, T=5003, cap=8192,
             dtype="fp32", ragged=True, fused=False),
        # one token of one short chat: launch latency
        dict(name="decode_short", kind="tree", fmt="bf16", B=1, Hq=8, Hkv=8, D=128, T=1, n=1999, window=0, sinks=0),
        # one token each of four 128k contexts, grouped heads, 8-bit cache: the cache is read once
        dict(name="decode_fp8_128k", kind="tree", fmt="mxfp8", B=4, Hq=32, Hkv=8, D=128, T=1, n=131072, window=0,
             sinks=0),
        # drafted trees verified against ragged 4-bit caches
        dict(name="tree_fp4_ragged", kind="tree", fmt="mxfp4", B=3, Hq=16, Hkv=4, D=128, T=29, n=50021, window=0,
             sinks=0),
        # a wide drafted tree over an 8-bit cache, D = 64, in a windowed layer with sinks
        dict(name="tree64_window", kind="tree", fmt="mxfp8", B=8, Hq=32, Hkv=8, D=64, T=64, n=40000, window=8192,
             sinks=5),
        # a short windowed layer
        dict(name="window_short", kind="window", op="fwd", B=2, Hq=4, Hkv=2, D=64, S=1003, window=256, sinks=4),
        # a windowed layer over a 128k sequence
        dict(name="window_128k", kind="window", op="fwd", B=1, Hq=8, Hkv=4, D=128, S=131072, window=4096, sinks=64),
        # gradients of an odd length with grouped heads
        dict(name="window_bwd_odd", kind="window", op="bwd", B=1, Hq=8, Hkv=2, D=64, S=5003, window=1000, sinks=4),
        # gradients of a training sequence
        dict(name="window_bwd_32k", kind="window", op="bwd", B=1, Hq=16, Hkv=4, D=128, S=32768, window=2048, sinks=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("cache", "tree", "tree", "window", "window"))
    D = rng.choice((64, 128, 128))
    Hkv = rng.choice((1, 2, 4, 8))
    if kind == "cache":
        fmt = rng.choice(("mxfp8", "mxfp4"))
        op = rng.choice(("write", "read"))
        B = rng.choice((1, 2, 3, 5, 16))
        T = _log(rng, 1, (1 << 20) // (B * Hkv))
        return dict(kind=kind, op=op, fmt=fmt, B=B, Hkv=Hkv, D=D, T=T, cap=(T + _log(rng, 1, 4096) + 15) // 16 * 16,
                    dtype=rng.choice(("bf16", "fp32")), ragged=rng.random() < 0.5, fused=rng.random() < 0.5)
    rep = rng.choice((1, 2, 4, 8))
    sinks = rng.choice((0, 1, 4, 100, 256))
    if kind == "tree":
        fmt = rng.choice(("mxfp8", "mxfp4", "bf16"))
        B = rng.choice((1, 2, 3, 7, 16))
        T = rng.choice((1, 1, 2, 7, 16, 33, 64))
        window = rng.choice((0, 0, _log(rng, 64, 16384)))
        return dict(kind=kind, fmt=fmt, B=B, Hq=Hkv * rep, Hkv=Hkv, D=D, T=T,
                    n=_log(rng, 1, min(131072, (1 << 21) // (B * Hkv))), window=window, sinks=sinks if window else 0)
    op = rng.choice(("fwd", "bwd"))
    B = rng.choice((1, 1, 2, 3))
    return dict(kind=kind, op=op, B=B, Hq=Hkv * rep, Hkv=Hkv, D=D,
                S=_log(rng, 128, (1 << (17 if op == "fwd" else 15)) // (B * Hkv)),
                window=_log(rng, 64, 4096), sinks=sinks)


# ------------------------------------------------------------------ formats (plain form)
def _split(x, fmt):
    """(codes uint8, scale bytes uint8) of x [..., D] in a microscaled format."""
    D = x.shape[-1]
    b = x.float().reshape(*x.shape[:-1], D // 32, 32)
    amax = b.abs().amax(-1)
    f, e = torch.frexp(amax)
    if fmt == "mxfp8":
        k = e - 9 + (f > _E4M3_MAX_F).int()
    else:
        k = e - 3 + (f > _E2M1_MAX_F).int()
    k = torch.where(amax > 0, k.clamp(-127, 127), torch.full_like(k, -127))
    y = torch.ldexp(b, -k[..., None])
    if fmt == "mxfp8":
        codes = y.to(torch.float8_e4m3fn).view(torch.uint8).reshape(x.shape)
    else:
        a = y.abs()
        c = (a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int() + \
            (a >= 3.5).int() + (a > 5.0).int()
        c = (c + 8 * torch.signbit(y).int()).reshape(*x.shape[:-1], D // 2, 2)
        codes = (c[..., 0] + 16 * c[..., 1]).to(torch.uint8)
    return codes, (k + 127).to(torch.uint8)


def _values(codes, scale, fmt):
    """fp32 values of cache rows (codes as stored, bf16 rows as they are)."""
    if fmt == "bf16":
        return codes.float()
    if fmt == "mxfp8":
        y = codes.view(torch.float8_e4m3fn).float()
    else:
        t = torch.tensor(_E2M1 + tuple(-x for x in _E2M1), device=codes.device)
        y = torch.stack((t[(codes & 15).int()], t[(codes >> 4).int()]), -1).reshape(*codes.shape[:-1],
                                                                                     2 * codes.shape[-1])
    y = y.reshape(*scale.shape, 32)
    return torch.ldexp(y, scale.int()[..., None] - 127).reshape(*scale.shape[:-1], 32 * scale.shape[-1])


# ------------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(1000003 * (seed + 1))


def _kv(g, shape, dtype, key):
    """K or V rows: a few head dimensions of K carry values several times the others', as trained keys do."""
    x = torch.empty(shape, device="cuda", dtype=dtype)
    for b in range(shape[0]):
        part = torch.randn(shape[1:], generator=g, device="cuda")
        if key:
            part[..., 3::29] *= 4.0
        x[b] = part.to(dtype)
    return x


def _ragged(B, top, seed, ragged=True):
    """One length per sequence, the first the longest."""
    r = torch.Generator().manual_seed(77 + seed)
    lo = max(1, top // 3)
    x = [top] + [int(torch.randint(lo, top + 1, (1,), generator=r)) for _ in range(B - 1)]
    return x if ragged else [top] * B


def _tree(B, T, seed):
    """Drafted trees: parent of each node (-1: a child of the last committed token), parents first."""
    r = torch.Generator().manual_seed(99 + seed)
    rows = []
    for _ in range(B):
        u = torch.rand(T, generator=r).tolist()
        p = torch.rand(T, generator=r).tolist()
        rows.append([i - 1 if u[i] < 0.5 else int(p[i] * (i + 1)) - 1 for i in range(T)])
    return rows


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _cache(g, c, n_rows):
    """Cache tensors of c's format with n_rows rows per sequence and head, all written."""
    out = []
    for key in (True, False):
        rows = _kv(g, (c["B"], c["Hkv"], n_rows, c["D"]), torch.bfloat16, key)
        if c["fmt"] == "bf16":
            out.append((rows, None))
            continue
        parts = [_split(rows[b], c["fmt"]) for b in range(c["B"])]
        out.append((torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])))
    return out


def _handle(st):
    from sequence_exact_attention_ring_b200 import KVCache

    return KVCache(st["fmt"], st["ck"], st["cv"], st["cks"], st["cvs"])


def prepare(case, seed):
    c, g = case, _gen(seed)
    if c["kind"] == "cache":
        return _prepare_cache(c, g, seed)
    if c["kind"] == "tree":
        return _prepare_tree(c, g, seed)
    B, Hq, Hkv, S, D = c["B"], c["Hq"], c["Hkv"], c["S"], c["D"]
    st = dict(c)
    st["q"] = _kv(g, (B, Hq, S, D), torch.bfloat16, False) * 1.5
    st["k"] = _kv(g, (B, Hkv, S, D), torch.bfloat16, True)
    st["v"] = _kv(g, (B, Hkv, S, D), torch.bfloat16, False)
    if c["op"] == "bwd":
        st["dout"] = _kv(g, (B, Hq, S, D), torch.bfloat16, False)
        st["out"], st["lse"] = _window_fwd(st)
    return st


def _prepare_cache(c, g, seed):
    B, Hkv, D, T, cap, fmt = c["B"], c["Hkv"], c["D"], c["T"], c["cap"], c["fmt"]
    st = dict(c)
    st["counts"] = _ragged(B, T, seed, c["ragged"])
    st["start"] = [(seed * 7 + 131 * b) % (cap - T + 1) for b in range(B)]
    st["d_counts"], st["d_start"] = _i32(st["counts"]), _i32(st["start"])
    if c["op"] == "write":
        dt = _DT[c["dtype"]]
        if c["fused"]:  # one projection's output [B, T, 2 Hkv D], seen as heads
            both = torch.empty(B, T, 2, Hkv, D, device="cuda", dtype=dt)
            for i in range(2):
                both[:, :, i] = _kv(g, (B, Hkv, T, D), dt, i == 0).transpose(1, 2)
            st["k_new"], st["v_new"] = both[:, :, 0].transpose(1, 2), both[:, :, 1].transpose(1, 2)
        else:
            st["k_new"], st["v_new"] = (_kv(g, (B, Hkv, T, D), dt, i == 0) for i in range(2))
        w = D if fmt == "mxfp8" else D // 2
        st["ck"], st["cv"] = (torch.zeros(B, Hkv, cap, w, dtype=torch.uint8, device="cuda") for _ in range(2))
        st["cks"], st["cvs"] = (torch.zeros(B, Hkv, cap, D // 32, dtype=torch.uint8, device="cuda") for _ in range(2))
    else:
        (st["ck"], st["cks"]), (st["cv"], st["cvs"]) = _cache(g, c, cap)
    if own:
        st["cache"] = _handle(st)
    return st


def _prepare_tree(c, g, seed):
    B, Hq, D, T = c["B"], c["Hq"], c["D"], c["T"]
    st = dict(c)
    st["lens"] = _ragged(B, c["n"], seed)
    st["parent_rows"] = _tree(B, T, seed)
    st["lengths"], st["parents"] = _i32(st["lens"]), _i32(st["parent_rows"])
    cap = (c["n"] + T + 15) // 16 * 16
    (st["ck"], st["cks"]), (st["cv"], st["cvs"]) = _cache(g, c, cap)
    # the query projection's output [B, T, Hq D], seen as heads
    st["q"] = (1.5 * torch.randn(B, T, Hq, D, generator=g, device="cuda")).to(torch.bfloat16).transpose(1, 2)
    if own:
        from sequence_exact_attention_ring_b200 import tree_workspace

        st["cache"] = _handle(st)
        st["ws"] = tree_workspace(st["q"], st["cache"])
    return st


# ---------------------------------------------------------------------------------- run
def run(state):
    if state["kind"] == "cache":
        return (_own_cache if own else _plain_cache)(state)
    if state["kind"] == "tree":
        return (_own_tree if own else _plain_tree)(state)
    if state["op"] == "fwd":
        return (_own_window_fwd if own else _window_fwd)(state)
    return (_own_window_bwd if own else _window_bwd)(state)


def _own_cache(st):
    from sequence_exact_attention_ring_b200 import cache_read, cache_write

    if st["op"] == "write":
        cache_write(st["cache"], st["k_new"], st["v_new"], st["d_start"], count=st["d_counts"])
    return cache_read(st["cache"], st["d_start"], st["T"], count=st["d_counts"], dtype=_DT[st["dtype"]])


def _plain_cache(st):
    B, Hkv, D, T, fmt = st["B"], st["Hkv"], st["D"], st["T"], st["fmt"]
    dt = _DT[st["dtype"]]
    pos = st["d_start"][:, None] + torch.arange(T, dtype=torch.int32, device="cuda")  # [B, T]
    live = torch.arange(T, device="cuda")[None] < st["d_counts"][:, None]
    b = torch.arange(B, device="cuda")[:, None].expand(B, T)[live]
    rows = pos[live].long()
    if st["op"] == "write":
        for new, codes, scale in ((st["k_new"], st["ck"], st["cks"]), (st["v_new"], st["cv"], st["cvs"])):
            c, s = _split(new, fmt)
            codes[b, :, rows] = c.transpose(1, 2)[live]
            scale[b, :, rows] = s.transpose(1, 2)[live]
    outs = []
    for codes, scale in ((st["ck"], st["cks"]), (st["cv"], st["cvs"])):
        x = torch.zeros(B, T, Hkv, D, dtype=dt, device="cuda")
        x[live] = _values(codes[b, :, rows], scale[b, :, rows], fmt).to(dt)
        outs.append(x.transpose(1, 2).contiguous())
    return tuple(outs)


def _own_tree(st):
    from sequence_exact_attention_ring_b200 import tree_attention

    return tree_attention(st["q"], st["cache"], st["lengths"], st["parents"], window=st["window"], sinks=st["sinks"],
                          workspace=st["ws"])


def _ancestors(parents):
    """[T, T] truth: node j is node i or one of its ancestors; and every node's depth [T]."""
    T = parents.shape[0]
    seen = torch.eye(T, dtype=torch.bool, device=parents.device)
    at = parents.long()
    me = torch.arange(T, device=parents.device)
    for _ in range(T - 1):
        ok = at >= 0
        seen[me[ok], at[ok]] = True
        at = torch.where(ok, parents.long()[at.clamp_min(0)], at)
    return seen, seen.sum(1) - 1


def _plain_tree(st):
    B, Hq, Hkv, T, D, W = st["B"], st["Hq"], st["Hkv"], st["T"], st["D"], st["window"]
    rep = Hq // Hkv
    out = torch.empty(B, Hq, T, D, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(B, Hq, T, dtype=torch.float32, device="cuda")
    for b in range(B):
        n = st["lens"][b]
        seen, depth = _ancestors(st["parents"][b])
        at = torch.cat((torch.arange(n, device="cuda"), n + depth))           # position of each key
        ok = torch.cat((torch.ones(T, n, dtype=torch.bool, device="cuda"), seen), 1)
        if W:
            ok &= (at[None] > (n + depth)[:, None] - W) | (at[None] < st["sinks"])
        use = ok.any(0).nonzero()[:, 0] if W else slice(0, n + T)
        ok = ok[:, use]
        k, v = (_values(x[b, :, :n + T][:, use], None if s is None else s[b, :, :n + T][:, use], st["fmt"])
                for x, s in ((st["ck"], st["cks"]), (st["cv"], st["cvs"])))
        q = st["q"][b].float().reshape(Hkv, rep, T, D)
        s = torch.matmul(q, k[:, None].transpose(-1, -2)) / math.sqrt(D)
        s = s.masked_fill(~ok, -math.inf)
        m = s.amax(-1, keepdim=True)
        p = torch.exp(s - m)
        l = p.sum(-1, keepdim=True)
        out[b] = (torch.matmul(p, v[:, None]) / l).reshape(Hq, T, D).to(torch.bfloat16)
        lse[b] = (m + torch.log(l)).reshape(Hq, T)
    return out, lse


def _own_window_fwd(st):
    from sequence_exact_attention_ring_b200 import window_attention

    return window_attention(st["q"], st["k"], st["v"], st["window"], st["sinks"])


def _own_window_bwd(st):
    from sequence_exact_attention_ring_b200 import window_attention_backward

    return window_attention_backward(st["q"], st["k"], st["v"], st["out"], st["lse"], st["dout"], st["window"],
                                     st["sinks"])


def _blocks(st):
    """Blocks of query rows with the keys that any of them sees, and the mask between them."""
    S, W, sinks = st["S"], st["window"], min(st["sinks"], st["S"])
    C = 512 if W <= 1024 else 2048
    for r0 in range(0, S, C):
        r1 = min(S, r0 + C)
        lo = max(0, r0 - W + 1)
        keys = torch.cat((torch.arange(min(sinks, lo), device="cuda"), torch.arange(lo, r1, device="cuda")))
        t = torch.arange(r0, r1, device="cuda")[:, None]
        yield r0, r1, keys, (keys <= t) & ((keys > t - W) | (keys < sinks))


def _window_fwd(st):
    B, Hq, Hkv, S, D = st["B"], st["Hq"], st["Hkv"], st["S"], st["D"]
    rep = Hq // Hkv
    out = torch.empty(B, Hq, S, D, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(B, Hq, S, dtype=torch.float32, device="cuda")
    for r0, r1, keys, ok in _blocks(st):
        q = st["q"][:, :, r0:r1].float().reshape(B, Hkv, rep, r1 - r0, D)
        k, v = st["k"][:, :, keys].float()[:, :, None], st["v"][:, :, keys].float()[:, :, None]
        s = (torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(D)).masked_fill(~ok, -math.inf)
        m = s.amax(-1, keepdim=True)
        p = torch.exp(s - m)
        l = p.sum(-1, keepdim=True)
        out[:, :, r0:r1] = (torch.matmul(p, v) / l).reshape(B, Hq, r1 - r0, D).to(torch.bfloat16)
        lse[:, :, r0:r1] = (m + torch.log(l)).reshape(B, Hq, r1 - r0)
    return out, lse


def _window_bwd(st):
    B, Hq, Hkv, S, D = st["B"], st["Hq"], st["Hkv"], st["S"], st["D"]
    rep = Hq // Hkv
    scale = 1 / math.sqrt(D)
    dq = torch.empty(B, Hq, S, D, dtype=torch.bfloat16, device="cuda")
    dk = torch.zeros(B, Hkv, S, D, dtype=torch.float32, device="cuda")
    dv = torch.zeros_like(dk)
    for r0, r1, keys, ok in _blocks(st):
        n = r1 - r0
        q, do, o = (st[x][:, :, r0:r1].float().reshape(B, Hkv, rep, n, D) for x in ("q", "dout", "out"))
        k, v = st["k"][:, :, keys].float()[:, :, None], st["v"][:, :, keys].float()[:, :, None]
        s = torch.matmul(q, k.transpose(-1, -2)) * scale
        p = torch.exp(s - st["lse"][:, :, r0:r1].reshape(B, Hkv, rep, n, 1)).masked_fill(~ok, 0.0)
        ds = p * (torch.matmul(do, v.transpose(-1, -2)) - (do * o).sum(-1, keepdim=True))
        dq[:, :, r0:r1] = (torch.matmul(ds, k) * scale).reshape(B, Hq, n, D).to(torch.bfloat16)
        dk.index_add_(2, keys, torch.matmul(ds.transpose(-1, -2), q).sum(2) * scale)
        dv.index_add_(2, keys, torch.matmul(p.transpose(-1, -2), do).sum(2))
    return dq, dk.to(torch.bfloat16), dv.to(torch.bfloat16)


# --------------------------------------------------------------------------------- work
def _seen_pairs(S, W, sinks):
    """(query, key) pairs of the causal window with sinks."""
    W, sinks = min(W, S), min(sinks, S)
    pairs = W * (W + 1) // 2 + (S - W) * W
    # sinks outside the window: token t >= W + u sees sink u < sinks besides its window
    top = min(sinks, S - W)
    return pairs + top * (S - W) - top * (top - 1) // 2


def work(case):
    c = case
    D, B = c["D"], c["B"]
    if c["kind"] == "window":
        pairs = _seen_pairs(c["S"], c["window"], c["sinks"])
        q, kv = B * c["Hq"] * c["S"], B * c["Hkv"] * c["S"]
        if c["op"] == "fwd":
            return {"bytes": 2 * D * (2 * q + 2 * kv) + 4 * q, "flops": 4 * D * B * c["Hq"] * pairs}
        return {"bytes": 2 * D * (4 * q + 4 * kv) + 4 * q, "flops": 10 * D * B * c["Hq"] * pairs}
    row = {"mxfp8": D + D // 32, "mxfp4": D // 2 + D // 32, "bf16": 2 * D}[c["fmt"]]
    if c["kind"] == "cache":
        n = sum(_ragged(B, c["T"], 0, c["ragged"])) * c["Hkv"] * 2
        wide = D * (2 if c["dtype"] == "bf16" else 4)
        full = B * c["T"] * c["Hkv"] * 2
        if c["op"] == "write":
            return {"bytes": n * (wide + 2 * row) + full * wide, "flops": 4 * D * n}
        return {"bytes": n * row + full * wide, "flops": 2 * D * n}
    T, W = c["T"], c["window"]
    keys = pairs = 0
    for n in _ragged(B, c["n"], 0):
        far = n if not W else min(n, W - 1 + min(c["sinks"], max(0, n - W + 1)))
        keys += far + T
        pairs += far * T + T * (T + 1) // 4
    return {"bytes": 2 * c["Hkv"] * keys * row + B * c["Hq"] * T * (4 * D + 4), "flops": 4 * D * c["Hq"] * pairs}


# -------------------------------------------------------------------------------- exact
def exact(case, seed):
    st = prepare(case, seed)
    if case["kind"] == "cache":
        return _exact_cache(st)
    if case["kind"] == "tree":
        return _exact_tree(st)
    return _exact_window(st)


def _exact_stored(x, fmt):
    """The value each element of x stands for once stored: a nearest multiple of the format's step, by its definition."""
    bits, least, top = (3, -6, 448.0) if fmt == "mxfp8" else (1, 0, 6.0)
    y = x.double().unflatten(-1, (-1, 32))
    big = y.abs().amax(-1, keepdim=True)
    k = torch.ceil(torch.log2((big / top).clamp_min(2.0 ** -127)))
    k = torch.where(big <= top * torch.exp2(k - 1), k - 1, k)
    k = torch.where(big > top * torch.exp2(k), k + 1, k).clamp_min(-127)
    unit = torch.exp2(k)
    y = y / unit
    e = torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -40)))
    e = torch.where(torch.exp2(e) > y.abs(), e - 1, e).clamp_min(least)
    step = torch.exp2(e - bits)
    return (torch.round(y / step) * step * unit).flatten(-2)


def _exact_decode(codes, scale, fmt):
    if fmt == "bf16":
        return codes.double()
    n = codes.int()
    if fmt == "mxfp4":
        n = torch.stack((n % 16, n // 16), -1).flatten(-2)
        sign, e, m, bias, bits = n // 8, (n // 2) % 4, n % 2, 1, 1
    else:
        sign, e, m, bias, bits = n // 128, (n // 8) % 16, n % 8, 7, 3
    one = (e > 0).double()
    y = (1 - 2 * sign.double()) * (one + m.double() / 2 ** bits) * torch.exp2(e.clamp_min(1).double() - bias)
    return (y.unflatten(-1, (-1, 32)) * torch.exp2(scale.double() - 127)[..., None]).flatten(-2)


def _exact_cache(st):
    B, Hkv, T, D = st["B"], st["Hkv"], st["T"], st["D"]
    if B * Hkv * T * D > 1 << 28:
        return None
    res = []
    for new, codes, scale in (("k_new", "ck", "cks"), ("v_new", "cv", "cvs")):
        x = torch.zeros(B, Hkv, T, D, dtype=torch.float64, device="cuda")
        for b, (n, s) in enumerate(zip(st["counts"], st["start"])):
            if st["op"] == "write":
                x[b, :, :n] = _exact_stored(st[new][b, :, :n], st["fmt"])
            else:
                x[b, :, :n] = _exact_decode(st[codes][b, :, s:s + n], st[scale][b, :, s:s + n], st["fmt"])
        res.append(x)
    return tuple(res)


def _exact_rows(q, k, v, ok):
    """Softmax attention in 64 bits of q [n, D] over k, v [L, D] where ok [n, L]."""
    s = (q.double() @ k.T) / math.sqrt(q.shape[-1])
    s = torch.where(ok, s, torch.full_like(s, -math.inf))
    lse = torch.logsumexp(s, -1)
    return torch.exp(s - lse[:, None]) @ v, lse


def _exact_tree(st):
    B, Hq, Hkv, T, D, W = st["B"], st["Hq"], st["Hkv"], st["T"], st["D"], st["window"]
    out = torch.empty(B, Hq, T, D, dtype=torch.float64, device="cuda")
    lse = torch.empty(B, Hq, T, dtype=torch.float64, device="cuda")
    for b, n in enumerate(st["lens"]):
        par = st["parent_rows"][b]
        ok = torch.zeros(T, n + T, dtype=torch.bool)
        for i in range(T):
            line = [i]
            while par[line[-1]] >= 0:
                line.append(par[line[-1]])
            line.reverse()  # root first: the node of depth d sits at position n + d
            at = n + len(line) - 1
            first = max(0, at - W + 1) if W else 0
            ok[i, min(first, n):n] = True
            ok[i, :min(st["sinks"] if W else 0, n)] = True
            for d, j in enumerate(line):
                ok[i, n + j] = n + d >= first or n + d < st["sinks"]
        ok = ok.cuda()
        for h in range(Hkv):
            k, v = (_exact_decode(x[b, h, :n + T], None if s is None else s[b, h, :n + T], st["fmt"])
                    for x, s in ((st["ck"], st["cks"]), (st["cv"], st["cvs"])))
            for r in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)):
                out[b, r], lse[b, r] = _exact_rows(st["q"][b, r], k, v, ok)
    return out, lse


def _exact_window(st):
    B, Hq, Hkv, S, D, W, sinks = (st[x] for x in ("B", "Hq", "Hkv", "S", "D", "window", "sinks"))
    rep, scale = Hq // Hkv, 1 / math.sqrt(D)
    bwd = st["op"] == "bwd"
    if not bwd:
        out = torch.empty(B, Hq, S, D, dtype=torch.float64, device="cuda")
        lse = torch.empty(B, Hq, S, dtype=torch.float64, device="cuda")
    else:
        dq = torch.empty(B, Hq, S, D, dtype=torch.float64, device="cuda")
        dk, dv = (torch.zeros(B, Hkv, S, D, dtype=torch.float64, device="cuda") for _ in range(2))
    step = 1024
    for r0 in range(0, S, step):
        r1 = min(S, r0 + step)
        first = max(0, r0 - W + 1)
        far = min(sinks, first)
        t = torch.arange(r0, r1, device="cuda")[:, None]
        u = torch.arange(r1, device="cuda")
        u = torch.cat((u[:far], u[first:]))[None]
        ok = (u <= t) & ((t - u < W) | (u < sinks))
        for b in range(B):
            for h in range(Hq):
                g = h // rep
                k = torch.cat((st["k"][b, g, :far], st["k"][b, g, first:r1])).double()
                v = torch.cat((st["v"][b, g, :far], st["v"][b, g, first:r1])).double()
                q = st["q"][b, h, r0:r1].double()
                if not bwd:
                    out[b, h, r0:r1], lse[b, h, r0:r1] = _exact_rows(q, k, v, ok)
                    continue
                do, o = st["dout"][b, h, r0:r1].double(), st["out"][b, h, r0:r1].double()
                p = torch.where(ok, torch.exp(scale * (q @ k.T) - st["lse"][b, h, r0:r1].double()[:, None]), 0.0)
                ds = p * (do @ v.T - (do * o).sum(1)[:, None])
                dq[b, h, r0:r1] = scale * (ds @ k)
                gk, gv = scale * (ds.T @ q), p.T @ do
                dk[b, g, :far] += gk[:far]
                dk[b, g, first:r1] += gk[far:]
                dv[b, g, :far] += gv[:far]
                dv[b, g, first:r1] += gv[far:]
    return (dq, dk, dv) if bwd else (out, lse)
