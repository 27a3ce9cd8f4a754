"""Timed cases of the 8-bit operators of a decoder layer: the paged 8-bit key/value cache (writing it, attention over
it), the residual + RMS norm, the 8-bit quantiser with SwiGLU, and the 8-bit block-scaled linear.

Each case names one operator and its sizes; `prepare` makes its inputs on the GPU, `run` is one call of the operator
(with `own`, the library's kernels through the Python binding; without, plain torch operations in fp32) and `exact` its
value in 64 bits.  Sizes are those of the 8B-class decoder the benchmark uses (hidden 4096, 32 query and 8 key/value
heads of 128, QKV output 6144, MLP width 12800), and generic ones around them.

Formulas (e4m3 is the OCP 8-bit format with a largest value of 448):
  append     cache page scale 2^e, e = clamp(ceil(log2(amax / 448)), -15, 8) over the page's tokens of one head (never
             below the scale the page already had for earlier tokens); code = e4m3(x / 2^e)
  attention  out_i = sum_j softmax_j(scale * q_i . k_j) v_j over positions j <= pos_i (j > pos_i - window)
  norm       h = x + r;  y = w * h / sqrt(mean(h^2) + eps)
  quantise   t = x, or silu(x[:, :K]) * x[:, K:];  per row and block of 128: s = max(amax, 2^-40) / 448,
             code = e4m3(t / s)
  linear     out[m, n] = sum_b sa[m, b] * sb[n / 128, b] * sum_{k in block b} a[m, k] * b[n, k]
"""
import math

import torch

own = False

FP8 = torch.float8_e4m3fn
H, HEADS, KV_HEADS, DIM, MLP, QKV = 4096, 32, 8, 128, 12800, 6144
EPS = 1e-6


def listed():
    return [
        # One generated token for each of 64 sequences: the cache write of every layer of every decode step.
        dict(name="append_decode", op="append", batch=64, rows=1, longest=700, heads=KV_HEADS, dim=DIM, page=64, seed=1),
        # Prompts of different lengths written at once, some continuing a page that is half full.
        dict(name="append_prompts", op="append", batch=5, rows=4000, longest=6000, heads=KV_HEADS, dim=DIM, page=64,
             seed=2),
        # The smallest call: a single user's token over a short cache; latency is all of it.
        dict(name="attend_one_user", op="attend", batch=1, rows=1, longest=777, heads=HEADS, kv_heads=KV_HEADS,
             dim=DIM, page=16, window=0, seed=3),
        # A serving batch: 48 users with caches from a few tokens to 16384; bound by reading the cache.
        dict(name="attend_batch", op="attend", batch=48, rows=1, longest=16384, heads=HEADS, kv_heads=KV_HEADS,
             dim=DIM, page=64, window=0, seed=4),
        # Prompts (one continuing a cached prefix) attended in one call; bound by the matrix cores.
        dict(name="attend_prompts", op="attend", batch=4, rows=4096, longest=6001, heads=HEADS, kv_heads=KV_HEADS,
             dim=DIM, page=64, window=0, seed=5),
        # The norm between two blocks of a decode step, fp16 out for a 4-bit linear.
        dict(name="norm_decode", op="norm", rows=3, width=H, fp8=False, seed=6),
        # The same for a prompt, 8 bits out for an 8-bit linear.
        dict(name="norm_prompt_8bit", op="norm", rows=8192, width=H, fp8=True, seed=7),
        # SwiGLU of a decode batch, 8 bits out for the down projection.
        dict(name="swiglu_decode", op="quant", rows=7, width=MLP, swiglu=True, seed=8),
        # SwiGLU of a prompt.
        dict(name="swiglu_prompt", op="quant", rows=4097, width=MLP, swiglu=True, seed=9),
        # The QKV projection of one token: bound by reading the weights.
        dict(name="linear_one_token", op="linear", M=1, K=H, N=QKV, seed=10),
        # The gate and up projections of a decode batch of odd size.
        dict(name="linear_batch", op="linear", M=37, K=H, N=2 * MLP, seed=11),
        # The same for a prompt: bound by the matrix cores.
        dict(name="linear_prompt", op="linear", M=4096, K=H, N=2 * MLP, seed=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "norm", "quant", "linear"])
    seed = rng.randrange(1 << 20)
    if op == "append":
        rows = rng.choice([1, _log(rng, 2, 3000)])
        batch = _log(rng, 1, 128 if rows == 1 else 6)
        return dict(op=op, batch=batch, rows=rows, longest=rows + _log(rng, 1, 3000), heads=rng.choice([1, 2, 4, 8, 32]),
                    dim=rng.choice([64, 128, 256]), page=rng.choice([16, 32, 64, 128]), seed=seed)
    if op == "attend":
        prompt = rng.random() < 0.4
        kv = rng.choice([1, 2, 4, 8])
        heads = kv * rng.choice([1, 2, 3, 4, 5, 8])
        rows = _log(rng, 2, 2500) if prompt else 1
        batch = _log(rng, 1, 4 if prompt else 40)
        longest = rows + _log(rng, 1, 2500) if prompt else _log(rng, 1, 12000)
        return dict(op=op, batch=batch, rows=rows, longest=longest, heads=min(heads, 32), kv_heads=kv if heads <= 32 else 4,
                    dim=rng.choice([64, 128, 256]) if heads <= 16 else rng.choice([64, 128]),
                    page=rng.choice([16, 32, 64, 128]), window=rng.choice([0, 0, 0, _log(rng, 16, 4096)]), seed=seed)
    if op == "norm":
        return dict(op=op, rows=_log(rng, 1, 6000), width=16 * _log(rng, 4, 512), fp8=rng.random() < 0.5, seed=seed)
    if op == "quant":
        return dict(op=op, rows=_log(rng, 1, 4000), width=16 * _log(rng, 4, 800), swiglu=rng.random() < 0.7, seed=seed)
    return dict(op=op, M=_log(rng, 1, 3000), K=16 * _log(rng, 8, 800), N=_log(rng, 100, 10000), seed=seed)


# ------------------------------------------------------------------ inputs ---

def _lengths(case):
    """(rows of each sequence in this call, its length in the cache with them): fixed by the case, spread over the
    range, the longest first."""
    rows, lens = [], []
    for i in range(case["batch"]):
        part = (i * 0.6180339887498949) % 1.0
        n = case["rows"] if i == 0 or case["rows"] == 1 else max(1, int(case["rows"] * part))
        whole = case["longest"] if i == 0 else max(n, int(case["longest"] * part))
        rows.append(n)
        lens.append(whole)
    return rows, lens


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _heavy(gen, *shape):
    """Activations as a trained model has them: nearly normal, with a few channels many times as large."""
    x = _randn(gen, *shape)
    big = torch.rand(shape[-1], generator=gen, device="cuda") < 0.01
    return torch.where(big, x * 12.0, x)


def _pages_of(x):
    """Quantises [pages, heads, page, dim] fp32 by page and head: codes and scale bytes."""
    amax = x.abs().amax(dim=(2, 3))
    byte = _scale_byte(amax)
    return (x / _pow2(byte)[:, :, None, None]).clamp(-448, 448).to(FP8), byte.to(torch.uint8)


def _pow2(byte):
    """2^(byte - 127) in fp32, exactly."""
    return (byte.to(torch.int32) << 23).view(torch.float32)


def _scale_byte(amax):
    """127 + clamp(ceil(log2(amax / 448)), -15, 8), from the bits of amax: 448 is 1.75 * 2^8."""
    e = ((amax.contiguous().view(torch.int32) + 0x1FFFFF) >> 23) - 127 - 8
    return e.clamp(-15, 8) + 127


def _cache(case, gen, lens, heads):
    """A cache pool with the sequences' pages in random order, and a table of them."""
    page, dim = case["page"], case["dim"]
    per = [-(-n // page) for n in lens]
    width, pages = max(per), sum(per) + 3
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros(len(lens), width, dtype=torch.int32)
    order_h, at = order.cpu(), 0
    for i, n in enumerate(per):
        table[i, :n] = order_h[at:at + n]
        at += n
    k = torch.empty(pages, heads, page, dim, dtype=FP8, device="cuda")
    v = torch.empty(pages, heads, dim, page, dtype=FP8, device="cuda")
    ks = torch.empty(pages, heads, dtype=torch.uint8, device="cuda")
    vs = torch.empty(pages, heads, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 27) // (heads * page * dim))
    for a in range(0, pages, step):
        n = min(step, pages - a)
        k[a:a + n], ks[a:a + n] = _pages_of(_heavy(gen, n, heads, page, dim).half().float())
        c, vs[a:a + n] = _pages_of(_randn(gen, n, heads, page, dim).half().float())
        v[a:a + n] = c.transpose(2, 3)
    return dict(k=k, v=v, k_scale=ks, v_scale=vs), table.cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + case["seed"])
    op = case["op"]
    if op in ("append", "attend"):
        rows, lens = _lengths(case)
        total = sum(rows)
        offsets = [0]
        for n in rows:
            offsets.append(offsets[-1] + n)
        heads = case["heads"] if op == "append" else case["kv_heads"]
        cache, table = _cache(case, gen, lens, heads)
        s = dict(op=op, cache=cache, table=table, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                 rows=None if case["rows"] == 1 else torch.tensor(offsets, dtype=torch.int32, device="cuda"),
                 longest=max(lens), most=max(rows), dim=case["dim"])
        if op == "append":
            width = heads * case["dim"]
            # keys and values as columns of the QKV projection's output
            s["qkv"] = torch.cat([_randn(gen, total, 2 * width), _heavy(gen, total, width),
                                  _randn(gen, total, width) * 1.5], dim=1).half()
            s["width"] = width
        else:
            s["q"] = _heavy(gen, total, case["heads"] * case["dim"]).mul_(0.7).half()
            s["window"], s["scale"] = case["window"], 1.0 / math.sqrt(case["dim"])
        return s
    if op == "norm":
        M, W = case["rows"], case["width"]
        return dict(op=op, x=_heavy(gen, M, W).half(), r=(_heavy(gen, M, W) * 3).half(),
                    w=(1 + 0.2 * _randn(gen, W)).half(), fp8=case["fp8"])
    if op == "quant":
        W = case["width"] * (2 if case["swiglu"] else 1)
        return dict(op=op, x=(_randn(gen, case["rows"], W) * 1.5).half(), swiglu=case["swiglu"])
    M, K, N = case["M"], case["K"], case["N"]
    kb, nb = -(-K // 128), -(-N // 128)
    a = (_randn(gen, M, K) * 110).clamp_(-448, 448).to(FP8)
    b = (_randn(gen, N, K) * 110).clamp_(-448, 448).to(FP8)
    sa = (torch.rand(M, kb, generator=gen, device="cuda") + 0.5) / 110
    sb = (torch.rand(nb, kb, generator=gen, device="cuda") + 0.5) / (110 * math.sqrt(K))
    return dict(op=op, a=a, sa=sa, b=b, sb=sb)


# -------------------------------------------------------------- plain forms ---

def _places(s):
    """For each row of the call: its sequence, and its position in it."""
    B = s["lens"].numel()
    lens = s["lens"].long()
    off = torch.arange(B + 1, device="cuda") if s["rows"] is None else s["rows"].long()
    total = (s["q"] if "q" in s else s["qkv"]).shape[0]
    t = torch.arange(total, device="cuda")
    b = torch.searchsorted(off, t, right=True) - 1
    first = lens - (off[1:] - off[:-1])
    return b, first[b] + t - off[b], first, off


def _plain_append(s):
    c, W, D = s["cache"], s["width"], s["dim"]
    heads, page = W // D, c["k"].shape[2]
    b, pos, first, off = _places(s)
    pid, at = s["table"].long()[b, pos // page], pos % page
    # pages that hold earlier tokens already: their old scale and how many tokens
    kept = first % page
    head_page = s["table"].long().gather(1, (first // page).clamp(max=s["table"].shape[1] - 1)[:, None])[:, 0]
    for name, lo in (("k", 2 * W), ("v", 3 * W)):
        x = s["qkv"][:, lo:lo + W].float().view(-1, heads, D)
        codes, scale = c[name], c[name + "_scale"]
        rows = codes if name == "k" else codes.transpose(2, 3)  # [pages, heads, page, dim]
        amax = torch.zeros(scale.shape, device="cuda").index_reduce_(0, pid, x.abs().amax(2), "amax")
        byte = _scale_byte(amax)
        had = torch.zeros(scale.shape[0], dtype=torch.bool, device="cuda").index_fill_(0, pid, True)
        new = torch.where(had[:, None], byte, scale.int())
        new = new.index_copy(0, head_page, torch.where(kept[:, None] > 0, torch.maximum(scale[head_page].int(), new[head_page]),
                                                       new[head_page]))
        old = rows[head_page].float()
        again = (old * _pow2(127 + scale[head_page].int() - new[head_page])[:, :, None, None]).to(FP8).float()
        earlier = torch.arange(page, device="cuda")[None, None, :, None] < kept[:, None, None, None]
        rows[head_page] = torch.where(earlier, again, old).to(FP8)
        rows[pid, :, at] = (x / _pow2(new[pid])[:, :, None]).clamp(-448, 448).to(FP8)
        scale.copy_(new)
    return c["k"], c["v"], c["k_scale"], c["v_scale"]


def _plain_attend(s):
    c, D = s["cache"], s["dim"]
    kvh, page = c["k"].shape[1], c["k"].shape[2]
    q = s["q"].float()
    heads = q.shape[1] // D
    G = heads // kvh
    b, pos, first, off = _places(s)
    B, L = s["table"].shape[0], s["table"].shape[1] * page
    t = s["table"].long()
    k = c["k"][t].float() * _pow2(c["k_scale"][t])[..., None, None]     # [B, pages, kvh, page, D]
    v = c["v"][t].float() * _pow2(c["v_scale"][t])[..., None, None]     # [B, pages, kvh, D, page]
    k = k.permute(0, 2, 4, 1, 3).reshape(B, kvh, D, L)
    v = v.permute(0, 2, 1, 4, 3).reshape(B, kvh, L, D)
    at = torch.arange(q.shape[0], device="cuda") - off[b]
    padded = torch.zeros(B, s["most"], heads, D, device="cuda")
    padded[b, at] = q.view(-1, heads, D)
    R = s["most"]
    padded = padded.view(B, R, kvh, G, D).permute(0, 2, 1, 3, 4).reshape(B, kvh, R * G, D)
    score = torch.matmul(padded, k).view(B, kvh, R, G, L) * s["scale"]
    where = first[:, None] + torch.arange(R, device="cuda")             # [B, R] positions
    j = torch.arange(L, device="cuda")
    seen = j <= where[..., None]
    if s["window"]:
        seen = seen & (j > where[..., None] - s["window"])
    score = score.masked_fill_(~seen[:, None, :, None, :], -torch.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -torch.inf, 0.0, top)
    p = score.sub_(top).exp_()
    p = p.div_(p.sum(-1, keepdim=True).clamp_min_(1e-30))
    out = torch.matmul(p.view(B, kvh, R * G, L), v).view(B, kvh, R, G, D)
    return out.permute(0, 2, 1, 3, 4).reshape(B, R, heads * D)[b, at].half()


def _plain_codes(y):
    M, W = y.shape
    nb = -(-W // 128)
    z = torch.nn.functional.pad(y, (0, nb * 128 - W)).view(M, nb, 128)
    amax = z.abs().amax(2).clamp_min(2.0 ** -40)
    codes = (z * (448.0 / amax)[..., None]).clamp(-448, 448).to(FP8)
    return codes.view(M, nb * 128)[:, :W].contiguous(), amax / 448.0


def _plain_norm(s):
    h = s["x"].float() + s["r"].float()
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * s["w"].float()
    return (*_plain_codes(y), h.half()) if s["fp8"] else (y.half(), h.half())


def _plain_quant(s):
    x = s["x"].float()
    if s["swiglu"]:
        g, u = x.chunk(2, 1)
        x = g / (1 + torch.exp(-g)) * u
    return _plain_codes(x)


def _plain_linear(s):
    M, K = s["a"].shape
    N = s["b"].shape[0]
    a = s["a"].float() * s["sa"].repeat_interleave(128, 1)[:, :K]
    b = s["b"].float() * s["sb"].repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    return torch.matmul(a, b.t()).half()


def run(state):
    s, op = state, state["op"]
    if not own:
        return {"append": _plain_append, "attend": _plain_attend, "norm": _plain_norm, "quant": _plain_quant,
                "linear": _plain_linear}[op](s)
    import w4a16_weight_only_amd as w4
    if op == "append":
        c, W = s["cache"], s["width"]
        w4.w4a16_kv_append(s["qkv"][:, 2 * W:3 * W], s["qkv"][:, 3 * W:], c, s["table"], s["lens"], rows=s["rows"])
        return c["k"], c["v"], c["k_scale"], c["v_scale"]
    if op == "attend":
        return w4.w4a16_attention(s["q"], s["cache"], s["table"], s["lens"], rows=s["rows"], scale=s["scale"],
                                  window=s["window"])
    if op == "norm":
        if s["fp8"]:
            (codes, scales), h = w4.w4a16_add_rmsnorm_fp8(s["x"], s["r"], s["w"], eps=EPS)
            return codes, scales, h
        return w4.w4a16_add_rmsnorm(s["x"], s["r"], s["w"], eps=EPS)
    if op == "quant":
        return w4.w4a16_quant_fp8(s["x"], act=w4.ACT_SWIGLU if s["swiglu"] else w4.ACT_NONE)
    return w4.w4a16_gemm_fp8(s["a"], s["sa"], s["b"], s["sb"])


# -------------------------------------------------------------- work, exact ---

def work(case):
    op = case["op"]
    if op in ("append", "attend"):
        rows, lens = _lengths(case)
        D = case["dim"]
        if op == "append":
            W = case["heads"] * D
            return dict(bytes=sum(rows) * W * (4 + 2), flops=sum(rows) * W * 4)
        window, kv, H_ = case["window"], case["kv_heads"], case["heads"]
        seen = pairs = 0
        for n, m in zip(rows, lens):
            first = m - n
            if window:
                pairs += sum(min(window, first + i + 1) for i in range(n))
                seen += min(m, n - 1 + window)
            else:
                pairs += n * first + n * (n + 1) // 2
                seen += m
        return dict(bytes=seen * kv * (2 * D + 2 / case["page"]) + sum(rows) * H_ * D * 4, flops=4.0 * pairs * H_ * D)
    if op == "norm":
        n = case["rows"] * case["width"]
        return dict(bytes=n * (6 + (1 + 4 / 128 if case["fp8"] else 2)) + case["width"] * 2, flops=6.0 * n)
    if op == "quant":
        n = case["rows"] * case["width"]
        return dict(bytes=n * ((4 if case["swiglu"] else 2) + 1 + 4 / 128), flops=n * (8.0 if case["swiglu"] else 3.0))
    M, K, N = case["M"], case["K"], case["N"]
    kb = -(-K // 128)
    return dict(bytes=M * K + N * K + M * N * 2 + 4 * kb * (M + -(-N // 128)), flops=2.0 * M * K * N)


def _exact_codes(y):
    """Values before their last rounding, and scales."""
    M, W = y.shape
    codes, scales = torch.empty_like(y), []
    for a in range(0, W, 128):
        blk = y[:, a:a + 128]
        s = torch.clamp(blk.abs().max(dim=1).values, min=2.0 ** -40) / 448
        codes[:, a:a + 128] = blk / s[:, None]
        scales.append(s)
    return codes, torch.stack(scales, 1)


def _exact_append(s):
    c, W, D = s["cache"], s["width"], s["dim"]
    heads, page = W // D, c["k"].shape[2]
    lens, table = s["lens"].tolist(), s["table"].tolist()
    off = list(range(len(lens) + 1)) if s["rows"] is None else s["rows"].tolist()
    got = []
    for name, lo in (("k", 2 * W), ("v", 3 * W)):
        codes = c[name].double() if name == "k" else c[name].double().transpose(2, 3).contiguous()
        scale = c[name + "_scale"].long()
        x = s["qkv"][:, lo:lo + W].double().view(-1, heads, D)
        for i, n in enumerate(lens):
            p = n - (off[i + 1] - off[i])
            while p < n:
                pid, a = table[i][p // page], p % page
                m = min(page - a, n - p)
                t = x[off[i + 1] - n + p:off[i + 1] - n + p + m].transpose(0, 1)     # [heads, m, D]
                e = torch.ceil(torch.log2(t.abs().amax((1, 2)) / 448)).clamp(-15, 8).long() + 127
                if a:
                    e = torch.maximum(e, scale[pid])
                    codes[pid, :, :a] = torch.ldexp(codes[pid, :, :a], (scale[pid] - e)[:, None, None])
                codes[pid, :, a:a + m] = torch.ldexp(t, (127 - e)[:, None, None])
                scale[pid] = e
                p += m
        got += [codes if name == "k" else codes.transpose(2, 3), scale.to(torch.uint8)]
    return got[0], got[2], got[1], got[3]


def _exact_attend(s):
    c, D = s["cache"], s["dim"]
    kvh, page = c["k"].shape[1], c["k"].shape[2]
    heads = s["q"].shape[1] // D
    lens = s["lens"].tolist()
    off = list(range(len(lens) + 1)) if s["rows"] is None else s["rows"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for i, n in enumerate(lens):
        ids = s["table"][i, :-(-n // page)].long()
        q = s["q"][off[i]:off[i + 1]].double().view(-1, heads, D)
        pos = torch.arange(n - q.shape[0], n, device="cuda")
        ks, vs = (torch.ldexp(torch.ones((), dtype=torch.float64, device="cuda"), c[x][ids].long() - 127)
                  for x in ("k_scale", "v_scale"))
        k = (c["k"][ids].double() * ks[..., None, None]).transpose(0, 1).reshape(kvh, -1, D)[:, :n]
        v = (c["v"][ids].double() * vs[..., None, None]).permute(1, 0, 3, 2).reshape(kvh, -1, D)[:, :n]
        gap = pos[:, None] - torch.arange(n, device="cuda")[None, :]
        hidden = gap < 0
        if s["window"]:
            hidden = hidden | (gap >= s["window"])
        for h in range(heads):
            kv = h // (heads // kvh)
            w = (q[:, h] @ k[kv].t().contiguous()) * s["scale"]
            w = torch.softmax(w.masked_fill(hidden, float("-inf")), dim=1)
            out[off[i]:off[i + 1], h * D:(h + 1) * D] = w @ v[kv]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "append":
        return _exact_append(s)
    if op == "attend":
        return _exact_attend(s)
    if op == "norm":
        h = s["x"].double() + s["r"].double()
        y = s["w"].double() * h / torch.sqrt((h * h).mean(dim=1, keepdim=True) + EPS)
        return (*_exact_codes(y), h) if s["fp8"] else (y, h)
    if op == "quant":
        x = s["x"].double()
        if s["swiglu"]:
            half = x.shape[1] // 2
            x = x[:, :half] * torch.sigmoid(x[:, :half]) * x[:, half:]
        return _exact_codes(x)
    M, K = s["a"].shape
    N = s["b"].shape[0]
    out = torch.zeros(M, N, dtype=torch.float64, device="cuda")
    column = torch.arange(N, device="cuda") // 128
    for i, k in enumerate(range(0, K, 128)):
        part = s["a"][:, k:k + 128].double() @ s["b"][:, k:k + 128].double().t()
        out += part * s["sa"][:, i].double()[:, None] * s["sb"][:, i].double()[column][None, :]
    return out
