"""Cases for the 4-bit microscaled operators and the quantised key/value cache.

Three paths, as a user's program calls them:

``quant``   a weight or a batch of activations is smoothed, quantised to blocks of 4-bit floating-point codes with one
            8-bit scale a block (MXFP4 or NVFP4), and read back as the values that the codes stand for.
``linear``  a batch of activations is smoothed and quantised, and multiplied with a weight that was quantised before.
``kv``      new tokens' keys and values are quantised into a paged cache, and a set of contexts is read back from it.

``run`` computes them in plain torch operations, or with the framework's own calls where ``own`` is true.  ``exact``
evaluates the operators' definition in 64 bits, rounding to 32 bits exactly where the definition rounds.
"""
import math

import torch

own = False

MX, NV = "mxfp4", "nvfp4"
BLOCK = {MX: 32, NV: 16}
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
FMAX = 3.4028234663852886e38


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one decode step of 16 requests: the down projection's input, latency counts
        dict(name="act_decode_mx", op="quant", side="act", fmt=MX, rows=16, K=11008, dt="bf16", out="f32", pad=0, smooth=True),
        # a calibration batch of an odd layer: odd rows, K that ends inside a block, rows cut out of a wider tensor
        dict(name="act_ragged_nv", op="quant", side="act", fmt=NV, rows=1021, K=1000, dt="f16", out="f32", pad=24, smooth=True),
        # a weight of a 7B MLP, quantised offline
        dict(name="weight_7b_nv", op="quant", side="weight", fmt=NV, rows=11008, K=4096, dt="bf16", out="bf16", pad=0, smooth=True),
        # the activations of a long prefill of a 70B layer
        dict(name="act_prefill_mx", op="quant", side="act", fmt=MX, rows=16384, K=8192, dt="bf16", out="bf16", pad=0, smooth=True),
        # one token through a 7B up projection: the weight is read once
        dict(name="linear_1_mx", op="linear", fmt=MX, M=1, N=11008, K=4096, dt="bf16", out="bf16", bias=False),
        # a decode batch through a 7B down projection with few weight rows
        dict(name="linear_100_nv", op="linear", fmt=NV, M=100, N=4096, K=11008, dt="bf16", out="f16", bias=True),
        # a prefill through the fused 7B query/key/value projection
        dict(name="linear_2048_mx", op="linear", fmt=MX, M=2048, N=12288, K=4096, dt="f16", out="bf16", bias=True),
        # a long prefill through one 70B MLP projection
        dict(name="linear_8192_nv", op="linear", fmt=NV, M=8192, N=28672, K=8192, dt="bf16", out="bf16", bias=False),
        # one decode step of 64 requests: a token each is written, and read back
        dict(name="kv_decode_int8", op="kv", fmt="int8", B=64, H=8, D=128, page=16, dt="bf16", old=0, new=1, back="new"),
        # odd heads and pages, a few tokens on top of contexts that are read back whole
        dict(name="kv_odd_int8", op="kv", fmt="int8", B=5, H=5, D=80, page=24, dt="f16", old=700, new=33, back="all"),
        # the prompts of 8 requests of uneven lengths
        dict(name="kv_prefill_fp8", op="kv", fmt="fp8", B=8, H=8, D=128, page=64, dt="bf16", old=0, new=2048, back="new"),
        # one decode step over long contexts, read back whole
        dict(name="kv_context_mx", op="kv", fmt="mxfp4", B=32, H=8, D=128, page=64, dt="bf16", old=4096, new=1, back="all"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quant", "linear", "kv"))
    dt = rng.choice(("bf16", "f16"))
    if op == "quant":
        K = _log(rng, 48, 16384)
        if rng.random() < 0.6:
            K = max(128, K // 128 * 128)
        rows = _log(rng, 1, max(2, min(16384, (1 << 26) // K)))
        return dict(op=op, side=rng.choice(("act", "weight")), fmt=rng.choice((MX, NV)), rows=rows, K=K,
                    dt=rng.choice(("bf16", "f16", "f32")), out=rng.choice(("bf16", "f16", "f32")), pad=rng.choice((0, 0, 8, 40)),
                    smooth=rng.random() < 0.8)
    if op == "linear":
        K = _log(rng, 64, 11008)
        N = _log(rng, 16, 16384)
        if rng.random() < 0.6:
            K, N = max(128, K // 128 * 128), max(16, N // 16 * 16)
        return dict(op=op, fmt=rng.choice((MX, NV)), M=_log(rng, 1, 4096), N=N, K=K, dt=dt, out=rng.choice(("bf16", "f16", "f32")),
                    bias=rng.random() < 0.5)
    H, B = rng.choice((1, 2, 5, 8, 32)), _log(rng, 1, 64)
    D = rng.choice((64, 72, 80, 96, 100, 128, 192, 256))
    most = max(2, min(8192, (1 << 26) // (B * H * D)))
    new = _log(rng, 1, most)
    return dict(op=op, fmt=rng.choice(("int8", "fp8", "mxfp4")), B=B, H=H, D=D, page=rng.choice((1, 16, 24, 64, 128)), dt=dt,
                old=rng.choice((0, _log(rng, 1, most))), new=new, back=rng.choice(("new", "all")))


def work(case):
    c = case
    if c["op"] == "quant":
        n, kp = c["rows"] * c["K"], -(-c["K"] // 32) * 32
        codes = c["rows"] * (kp // 2 + kp // BLOCK[c["fmt"]])
        # the input is read; codes and scales are written and read again; the values are written
        return {"bytes": n * (DT[c["dt"]].itemsize + DT[c["out"]].itemsize) + 2 * codes + 4 * c["K"], "flops": 4 * n}
    if c["op"] == "linear":
        M, N, kp = c["M"], c["N"], -(-c["K"] // 32) * 32
        per = kp // 2 + kp // BLOCK[c["fmt"]]
        # activations and packed weights are read, the output is written; the packed activations stay on the chip
        return {"bytes": M * c["K"] * DT[c["dt"]].itemsize + N * per + M * N * DT[c["out"]].itemsize + 4 * c["K"],
                "flops": 2 * M * N * c["K"]}
    lens = _lengths(c)
    new, back = sum(n for _, n in lens), sum((o if c["back"] == "all" else 0) + n for o, n in lens)
    row = 2 * c["H"] * c["D"]
    per = {"int8": 1 + 4 / c["D"], "fp8": 1 + 4 / c["D"], "mxfp4": 0.5 + 1 / 32}[c["fmt"]]
    # new tokens are read and their codes written; the contexts' codes are read and their values written
    return {"bytes": row * (new * (2 + per) + back * (per + 2)), "flops": 4 * row * (new + back)}


# ---------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _acts(g, M, K, dt, pad=0):
    """Activations with a few channels far above the rest, as the smoothing meets them; rows may be cut out of wider ones."""
    x = torch.randn(M, K + pad, generator=g, device="cuda")
    hot = torch.randint(0, K + pad, (max(1, K // 200),), generator=g, device="cuda")
    x[:, hot] *= 30.0
    return x.to(dt)[:, :K]


def _smoothing(x, w_col):
    """max|X_j|^0.5 / max|W_j|^0.5 with both statistics clamped at 1e-5."""
    a = x.float().abs().amax(0).clamp_min(1e-5)
    return (a.double().sqrt() / w_col.clamp_min(1e-5).double().sqrt()).float()


def _lengths(c):
    """(tokens held, tokens written) of each sequence: uneven, the same for every seed."""
    out = []
    for b in range(c["B"]):
        f = 1.0 - 0.85 * ((b * 7) % c["B"]) / max(1, c["B"])
        out.append((int(c["old"] * f), max(1, int(c["new"] * f))))
    return out


def prepare(case, seed):
    c, g = case, _gen(seed)
    if c["op"] == "quant":
        dt = DT[c["dt"]]
        if c["side"] == "act":
            x = _acts(g, c["rows"], c["K"], dt, c["pad"])
            col = 0.02 * (1 + torch.rand(c["K"], generator=g, device="cuda"))
            s = _smoothing(x, col)
            top = x.float().abs().amax(0) / s if c["smooth"] else x.float().abs().amax(0)
        else:
            x = (0.02 * torch.randn(c["rows"], c["K"], generator=g, device="cuda")).to(dt)
            s = 0.5 + 3.0 * torch.rand(c["K"], generator=g, device="cuda")
            top = x.float().abs().amax(0) * (s if c["smooth"] else 1.0)
        st = dict(c=c, x=x, s=s if c["smooth"] else None, g=_tensor_scale(top) if c["fmt"] == NV else None)
        # a user's program keeps the buffers that codes, scales and values are written to
        st["q"], st["sf"] = _fp4_buffers(c["rows"], c["K"], c["fmt"])
        st["y"] = torch.empty(c["rows"], c["K"], dtype=DT[c["out"]], device="cuda")
        return st
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        x = _acts(g, M, K, DT[c["dt"]])
        w = 0.02 * torch.randn(N, K, generator=g, device="cuda")
        s = _smoothing(x, w.abs().amax(0))
        ga = gw = None
        if c["fmt"] == NV:
            ga, gw = _tensor_scale(x.float().abs().amax(0) / s), _tensor_scale(w.abs().amax(0) * s)
        sf, code = _quant_plain(w.mul_(s), c["fmt"], gw)
        del w
        st = dict(c=c, x=x, s=s, ga=ga, gw=gw, wq=_pack(code), wsf=_tile_scales(sf, c["fmt"]))
        st["bias"] = torch.randn(N, generator=g, device="cuda").to(DT[c["out"]]) if c["bias"] else None
        st["q"], st["sf"] = _fp4_buffers(M, K, c["fmt"])
        st["y"] = torch.empty(M, N, dtype=DT[c["out"]], device="cuda")
        return st
    B, H, D, page = c["B"], c["H"], c["D"], c["page"]
    lens = _lengths(c)
    pages = [-(-(o + n) // page) for o, n in lens]
    P = sum(pages) + 3
    order = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(B, max(pages), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = order[at:at + n]
        at += n
    rows, sb = _kv_bytes(c["fmt"], D)
    st = dict(c=c, table=table)
    T = sum(n for _, n in lens)
    # keys and values lie beside the queries in the output of one projection
    qkv = torch.randn(T, 3 * H * D, generator=g, device="cuda")
    qkv[:, ::61] *= 8.0
    qkv = qkv.to(DT[c["dt"]])
    st["k"], st["v"] = (qkv[:, i * H * D:(i + 1) * H * D].unflatten(1, (H, D)) for i in (1, 2))
    for n in "kv":  # what the contexts hold already
        if c["fmt"] == "int8":
            st[n + "c"] = torch.randint(-127, 128, (P, page, H, rows), generator=g, device="cuda", dtype=torch.int8)
        elif c["fmt"] == "fp8":
            st[n + "c"] = torch.randint(0, 127, (P, page, H, rows), generator=g, device="cuda", dtype=torch.uint8)
        else:
            st[n + "c"] = torch.randint(0, 256, (P, page, H, rows), generator=g, device="cuda", dtype=torch.uint8)
        if c["fmt"] == "mxfp4":
            st[n + "s"] = torch.randint(120, 130, (P, page, H, sb), generator=g, device="cuda", dtype=torch.uint8)
        else:
            st[n + "s"] = 0.01 + 0.05 * torch.rand(P, page, H, generator=g, device="cuda")
    pos = torch.cat([torch.arange(o, o + n) for o, n in lens]).cuda()
    seq = torch.repeat_interleave(torch.arange(B), torch.tensor([n for _, n in lens])).cuda()
    st["slots"] = table[seq, pos // page].long() * page + pos % page
    first = [0 if c["back"] == "all" else o for o, _ in lens]
    span = [o + n - f for (o, n), f in zip(lens, first)]
    st["starts"] = torch.tensor(first, dtype=torch.int32).cuda()
    st["cu"] = torch.tensor([sum(span[:b]) for b in range(B + 1)], dtype=torch.int32).cuda()
    st["ko"], st["vo"] = (torch.empty(sum(span), H, D, dtype=DT[c["dt"]], device="cuda") for _ in "kv")
    # where each row that is read back lies: an index that a program without a paged read keeps
    pos = torch.cat([torch.arange(f, f + n) for f, n in zip(first, span)]).cuda()
    seq = torch.repeat_interleave(torch.arange(B), torch.tensor(span)).cuda()
    st["back"] = table[seq, pos // page].long() * page + pos % page
    return st


# ---------------------------------------------------------------- formats, in plain operations
def _tensor_scale(top):
    return (top.max() / 2688.0).reshape(1)


def _fp4_buffers(rows, K, fmt):
    kp = -(-K // 32) * 32
    n = -(-rows // 128) * -(-(kp // BLOCK[fmt]) // 4) * 512
    return torch.empty(rows, kp // 2, dtype=torch.uint8, device="cuda"), torch.empty(n, dtype=torch.uint8, device="cuda")


def _kv_bytes(fmt, D):
    return (-(-D // 32) * 16, -(-D // 32)) if fmt == "mxfp4" else (-(-D // 16) * 16, 4)


def _recip(v):
    """1/v, the largest finite number where that overflows, 0 for v = 0."""
    return torch.where(v > 0, (1.0 / v).clamp_max(FMAX), torch.zeros_like(v))


def _round_e2m1(a):
    """Index of the nearest of E2M1 for a >= 0, ties to the even index, 7 beyond."""
    i = (a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    return i


def _e4m3(v):
    return v.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).float()


def _blocks(x, fmt):
    """[rows, K] in 32 bits -> [rows, blocks, block], zeros behind K up to a multiple of 32."""
    K = x.shape[1]
    x = torch.nn.functional.pad(x, (0, -K % 32))
    return x.unflatten(1, (-1, BLOCK[fmt]))


def _quant_plain(x, fmt, g):
    """Scale bytes [rows, blocks] and codes [rows, K'] of 32-bit values."""
    x = _blocks(x, fmt)
    m = x.abs().amax(2)
    if fmt == MX:
        sf = ((m.view(torch.int32) >> 23) - 2).clamp_min(0)
        inv = ((254 - sf) << 23).view(torch.float32)
        sf = sf.to(torch.uint8)
    else:
        c = _recip(g) * torch.full_like(g, 1.0 / 6.0)
        v = _e4m3(m * c)
        sf = v.to(torch.float8_e4m3fn).view(torch.uint8)
        inv = _recip(v * g)
    x = x * inv[..., None]
    code = _round_e2m1(x.abs()) + (x < 0).to(torch.uint8) * 8
    return sf, code.flatten(1)


def _scale_values(sf, fmt, g):
    if fmt == MX:
        return torch.ldexp(torch.ones((), device="cuda"), sf.to(torch.int32) - 127)
    v = sf.view(torch.float8_e4m3fn).float()
    return v if g is None else v * g


def _code_values(code):
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")
    return lut[code.to(torch.int32)]


def _values(code, sf, fmt, g):
    return (_code_values(code).unflatten(1, (-1, BLOCK[fmt])) * _scale_values(sf, fmt, g)[..., None]).flatten(1)


def _pack(code):
    return code[:, 0::2] | (code[:, 1::2] << 4)


def _unpack(q):
    return torch.stack((q & 15, q >> 4), dim=-1).flatten(-2)


def _tile_scales(sf, fmt):
    """[rows, blocks] scale bytes -> tiles of 128 rows x 4 blocks, row r of a tile at 16 (r % 32) + 4 (r / 32)."""
    sf = torch.nn.functional.pad(sf, (0, -sf.shape[1] % 4, 0, -sf.shape[0] % 128))
    return sf.unflatten(1, (-1, 4)).unflatten(0, (-1, 4, 32)).permute(0, 3, 2, 1, 4).flatten()


def _untile_scales(t, rows, K, fmt):
    n = -(-K // 32) * 32 // BLOCK[fmt]
    t = t.view(-(-rows // 128), -(-n // 4), 32, 4, 4).permute(0, 3, 2, 1, 4)
    return t.reshape(t.shape[0] * 128, -1)[:rows, :n]


# ---------------------------------------------------------------- one pass
def run(state):
    c = state["c"]
    if own:
        return _run_own(state, c)
    if c["op"] == "quant":
        x = state["x"].float()
        if state["s"] is not None:
            x = x * (_recip(state["s"]) if c["side"] == "act" else state["s"])
        sf, code = _quant_plain(x, c["fmt"], state["g"])
        return _values(code, sf, c["fmt"], state["g"])[:, :c["K"]].to(DT[c["out"]])
    if c["op"] == "linear":
        sf, code = _quant_plain(state["x"].float() * _recip(state["s"]), c["fmt"], state["ga"])
        x = _values(code, sf, c["fmt"], None)
        wsf = _untile_scales(state["wsf"], c["N"], c["K"], c["fmt"])
        y = x @ _values(_unpack(state["wq"]), wsf, c["fmt"], None).t()
        if c["fmt"] == NV:
            y = y * (state["ga"] * state["gw"])
        if c["bias"]:
            y = y + state["bias"].float()
        return y.to(DT[c["out"]])
    return tuple(_kv_plain(state, c, n) for n in "kv")


def _kv_plain(st, c, n):
    D, x = c["D"], st[n].float()
    cache, scale = st[n + "c"].flatten(0, 1), st[n + "s"].flatten(0, 1)
    if c["fmt"] == "mxfp4":
        sf, code = _quant_plain(x.flatten(0, 1), MX, None)
        cache[st["slots"]] = _pack(code).unflatten(0, x.shape[:2])
        scale[st["slots"]] = sf.unflatten(0, x.shape[:2])
        q, sf = cache[st["back"]], scale[st["back"]]
        v = _values(_unpack(q).flatten(0, 1), sf.flatten(0, 1), MX, None)
        return v[:, :D].unflatten(0, q.shape[:2]).to(DT[c["dt"]])
    top = 127.0 if c["fmt"] == "int8" else 448.0
    a = x.abs().amax(2)
    a = a / torch.full_like(a, top)  # by a tensor: a division by a number is a product with its rounded inverse
    x = x * _recip(a)[..., None]
    if c["fmt"] == "int8":
        q = x.round().clamp(-127, 127).to(torch.int8)
    else:
        q = x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    cache[st["slots"]] = torch.nn.functional.pad(q, (0, cache.shape[-1] - D))
    scale[st["slots"]] = a
    q = cache[st["back"]][..., :D]
    q = q.float() if c["fmt"] == "int8" else q.contiguous().view(torch.float8_e4m3fn).float()
    return (q * scale[st["back"]][..., None]).to(DT[c["dt"]])


def _run_own(st, c):
    import w8a8_post_quantization_calib_b200 as sq
    fmt = {MX: sq.MXFP4, NV: sq.NVFP4}.get(c["fmt"])
    if c["op"] == "quant":
        quantise = sq.smooth_quant_act_fp4 if c["side"] == "act" else sq.quant_weight_fp4
        quantise(st["x"], st["s"], fmt, st["q"], st["sf"], g=st["g"])
        sq.dequant_fp4(st["q"], st["sf"], fmt, st["y"], g=st["g"])
        return st["y"]
    if c["op"] == "linear":
        sq.smooth_quant_act_fp4(st["x"], st["s"], fmt, st["q"], st["sf"], g=st["ga"])
        sq.linear_fp4(st["q"], st["sf"], st["wq"], st["wsf"], fmt, st["y"], bias=st["bias"], g_act=st["ga"], g_w=st["gw"])
        return st["y"]
    fmt = {"int8": sq.KV_INT8, "fp8": sq.KV_FP8, "mxfp4": sq.KV_MXFP4}[c["fmt"]]
    sq.kv_cache_write(st["k"], st["v"], st["slots"], fmt, st["kc"], st["ks"], st["vc"], st["vs"])
    sq.kv_cache_read(fmt, st["kc"], st["ks"], st["vc"], st["vs"], st["table"], st["cu"], st["ko"], st["vo"], starts=st["starts"])
    return st["ko"], st["vo"]


# ---------------------------------------------------------------- the definition, in 64 bits
def _r32(v):
    return v.float().double()


def _inv64(v):
    """fl32(1/v), the largest finite number where that overflows, 0 for v = 0 (the quotient rounds once: 53 >= 2 * 24 + 2)."""
    return torch.where(v > 0, (1.0 / v).float().clamp_max(FMAX).double(), torch.zeros_like(v))


def _nearest64(v, points):
    """Nearest of the ascending points for v >= 0, ties to the even index, the last one beyond."""
    p = torch.tensor(points, dtype=torch.float64, device=v.device)
    hi = torch.searchsorted(p, v.contiguous()).clamp_max(len(points) - 1)
    lo = (hi - 1).clamp_min(0)
    below, above = v - p[lo], p[hi] - v
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    return torch.where(up | (hi == 0), p[hi], p[lo])


E4M3 = tuple(m / 512.0 for m in range(8)) + tuple((1 + m / 8.0) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)
                                                  if (e, m) != (15, 7))


def _fp4_exact(x, fmt, g, with_g=True):
    """The values of [rows, K] after quantisation; without the tensor's scale where with_g is false."""
    rows, K = x.shape
    n = BLOCK[fmt]
    pad = torch.zeros(rows, -(-K // n) * n, dtype=torch.float64, device=x.device)
    pad[:, :K] = x
    b = pad.view(rows, -1, n)
    m = b.abs().amax(2)
    if fmt == MX:
        e = torch.where(m > 0, torch.frexp(m).exponent.double() - 1, torch.full_like(m, -200.0)) - 2
        scale = inner = torch.exp2(e.clamp_min(-127.0))
        v = b / inner[..., None]
    else:
        g = g.double()
        c = _r32(_inv64(g) * float(torch.tensor(1.0 / 6.0)))
        inner = _nearest64(_r32(m * c), E4M3)
        scale = _r32(inner * g)
        v = _r32(b * _inv64(scale)[..., None])
    v = _nearest64(v.abs(), E2M1) * torch.sign(v)
    out = v * (scale if with_g else inner)[..., None]
    return out.reshape(rows, -1)[:, :K]


def exact(case, seed):
    st, c = prepare(case, seed), case
    if c["op"] == "quant":
        x = st["x"].double()
        if st["s"] is not None:
            s = st["s"].double()
            x = _r32(x * (_inv64(s) if c["side"] == "act" else s))
        return _fp4_exact(x, c["fmt"], st["g"])
    if c["op"] == "linear":
        x = _fp4_exact(_r32(st["x"].double() * _inv64(st["s"].double())), c["fmt"], st["ga"], with_g=False)
        q = st["wq"].long()
        code = torch.empty(c["N"], 2 * q.shape[1], dtype=torch.float64, device=q.device)
        lut = torch.tensor([v * f for f in (1.0, -1.0) for v in E2M1], dtype=torch.float64, device=q.device)
        code[:, 0::2], code[:, 1::2] = lut[q % 16], lut[q // 16]
        del q
        n, B = code.shape[1] // BLOCK[c["fmt"]], BLOCK[c["fmt"]]
        r, k = torch.arange(c["N"], device="cuda")[:, None], torch.arange(n, device="cuda")[None, :]
        sf = st["wsf"][((r // 128) * -(-n // 4) + k // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + k % 4].long()
        if c["fmt"] == MX:
            sf = torch.exp2(sf.double() - 127)
        else:
            sf = torch.tensor(E4M3 + (math.nan,), dtype=torch.float64, device="cuda")[sf]
        code.view(c["N"], n, B).mul_(sf[..., None])
        y = x @ code[:, :c["K"]].t()
        if c["fmt"] == NV:
            y = y * (st["ga"].double() * st["gw"].double())
        return y + st["bias"].double() if c["bias"] else y
    return tuple(_kv_exact(st, c, n) for n in "kv")


def _kv_exact(st, c, n):
    """Every row that is read back: the new tokens' quantised values, or what the cache held."""
    D, H, f = c["D"], c["H"], c["fmt"]
    cache, scale = st[n + "c"].reshape(-1, H, st[n + "c"].shape[-1]), st[n + "s"].flatten(0, 1)
    new = torch.full((cache.shape[0],), -1, dtype=torch.long, device="cuda")
    new[st["slots"]] = torch.arange(st["slots"].numel(), device="cuda")
    which = new[st["back"]]
    x = st[n].double()
    if f == "mxfp4":
        fresh = _fp4_exact(x.reshape(-1, D), MX, None).view(-1, H, D)
        q = cache[st["back"]].long()
        lut = torch.tensor([v * t for t in (1.0, -1.0) for v in E2M1], dtype=torch.float64, device="cuda")
        held = torch.stack((lut[q % 16], lut[q // 16]), -1).flatten(-2)
        held = (held.unflatten(-1, (-1, 32)) * torch.exp2(scale[st["back"]].double() - 127)[..., None]).flatten(-2)[..., :D]
    else:
        a = x.abs().amax(2)
        a = _r32(a / torch.full_like(a, 127.0 if f == "int8" else 448.0))
        v = _r32(x * _inv64(a)[..., None])
        v = torch.round(v).clamp(-127, 127) if f == "int8" else _nearest64(v.abs(), E4M3) * torch.sign(v)
        fresh = v * a[..., None]
        q = cache[st["back"]][..., :D].long()
        held = q.double() if f == "int8" else torch.tensor(E4M3, dtype=torch.float64, device="cuda")[q]
        held = held * scale[st["back"]].double()[..., None]
    return torch.where((which >= 0)[:, None, None], fresh[which.clamp_min(0)], held)
