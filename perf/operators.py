"""What the operators around the paged FP4 cache are measured on.

Four operators of one serving step: pages and slots for new tokens
(page_plan), the residual sum with its root-mean-square norm cast to FP8
blocks (rms_norm_fp8), rotary positions (rope), and attention over the pages
of a cache held in 4 bits (paged_decode_fp4).  With `own` false `run`
computes them in plain torch operations; with `own` true it makes the calls
that a program makes of fp4_kv_cache_sparse_gb300.
"""
import math

import torch

own = False

PAGE = 64
DIM = 512
REC = 288
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # One sequence, one token, few heads: the latency of a single call.
        dict(name="attn_b1_h16_l700", op="attn", batch=1, s=1, h=16, lmin=700, lmax=700, window=0, sinks=0),
        # An ordinary batch of 64-head decode steps over ragged lengths.
        dict(name="attn_b64_h64_l8k", op="attn", batch=64, s=1, h=64, lmin=1024, lmax=8192, window=0, sinks=0),
        # Long contexts, few heads on this GPU: the bytes of the cache.
        dict(name="attn_b32_h16_l64k", op="attn", batch=32, s=1, h=16, lmin=65536, lmax=65536, window=0, sinks=0),
        # Speculative decode (two tokens), all heads, window and sinks.
        dict(name="attn_b32_s2_h128_w4k", op="attn", batch=32, s=2, h=128, lmin=6000, lmax=32768, window=4096, sinks=128),
        # Odd head count, three tokens, short and empty sequences, small window.
        dict(name="attn_b7_s3_h24_w1000", op="attn", batch=7, s=3, h=24, lmin=0, lmax=5001, window=1000, sinks=4),
        # One decode step's latents: few rows, latency.
        dict(name="norm_64x512", op="norm", n=64, d=512, dtype="bf16", residual=False),
        # A prefill chunk's hidden states with the residual stream.
        dict(name="norm_8191x8192_res", op="norm", n=8191, d=8192, dtype="bf16", residual=True),
        # Latents of a long prefill in half precision.
        dict(name="norm_200000x512_fp16", op="norm", n=200000, d=512, dtype="fp16", residual=False),
        # The rotary tail of a step's queries (64 of 512 dims), in place.
        dict(name="rope_256x128_tail", op="rope", n=256, h=128, d=512, off=448, rd=64, dtype="bf16", layout="interleaved",
             scaling="none", maxpos=131072, inplace=True),
        # A prefill chunk's heads in the half layout, scaled for long contexts.
        dict(name="rope_8000x32_half", op="rope", n=8000, h=32, d=128, off=0, rd=128, dtype="fp16", layout="half",
             scaling="yarn", maxpos=1048576, inplace=False),
        # One decode step of 256 requests: a token each.
        dict(name="plan_b256_decode", op="plan", batch=256, nmin=1, nmax=1, cmax=131072, gone=0),
        # Chunked prefill beside decodes, some requests ending.
        dict(name="plan_b1000_prefill", op="plan", batch=1000, nmin=0, nmax=512, cmax=32768, gone=20),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "norm", "rope", "plan"])
    if op == "attn":
        h = rng.choice([16, 16, 32, 64, 128, rng.randrange(1, 129)])
        s = rng.choice([1, 1, 2, rng.randrange(1, 7)])
        batch = _log(rng, 1, 128)
        # No costlier than the largest listed cases, in bytes and in products.
        most = min(32 * 65536 // batch, 64 * 8192 * 64 // (batch * s * h), 65536)
        lmax = _log(rng, min(200, most), most)
        window = rng.choice([0, 0, _log(rng, 16, 8192)])
        return dict(op=op, batch=batch, s=s, h=h, lmin=rng.choice([0, lmax // 2, lmax]), lmax=lmax, window=window,
                    sinks=rng.choice([0, 4, rng.randrange(0, 300)]) if window else 0)
    if op == "norm":
        d = 32 * _log(rng, 1, 256)
        t = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        return dict(op=op, n=_log(rng, 1, max(2, (30_000_000 if t == "fp32" else 60_000_000) // d)), d=d, dtype=t,
                    residual=rng.random() < 0.5)
    if op == "rope":
        rd = 2 * rng.choice([16, 32, 32, 64, rng.randrange(4, 65)])
        d = rd + rng.choice([0, 0, 448, 2 * rng.randrange(0, 100)])
        h = rng.choice([1, 8, 32, 128, rng.randrange(1, 129)])
        return dict(op=op, n=_log(rng, 1, max(2, 30_000_000 // (h * d))), h=h, d=d, off=rng.choice([0, d - rd]), rd=rd,
                    dtype=rng.choice(["bf16", "fp16", "fp32"]), layout=rng.choice(["interleaved", "half"]),
                    scaling=rng.choice(["none", "linear", "yarn"]), maxpos=_log(rng, 1000, 1 << 20),
                    inplace=rng.random() < 0.3)
    batch = _log(rng, 1, 2000)
    nmin = rng.choice([0, 1])
    return dict(op=op, batch=batch, nmin=nmin, nmax=nmin + _log(rng, 1, 250000 // batch), cmax=_log(rng, 64, 65536),
                gone=rng.choice([0, batch // 10]))


# ---------------------------------------------------------------- inputs


def _encode_fp4(x):
    """fp32 [n, 512] -> 288-byte records: amax/6 per 16 values as e4m3, e2m1 data, even dim in the low nibble."""
    n = x.shape[0]
    b = x.view(n, 32, 16)
    sc = (b.abs().amax(-1) / 6.0).to(torch.float8_e4m3fn)
    y = b / sc.float().clamp_min(2.0 ** -9).unsqueeze(-1)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
    code = torch.bucketize(y.abs(), edges).to(torch.uint8) | ((y < 0).to(torch.uint8) << 3)
    code = code.view(n, 256, 2)
    return torch.cat([code[..., 0] | (code[..., 1] << 4), sc.view(torch.uint8)], 1)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    gc = torch.Generator().manual_seed(seed)
    c = case

    def randn(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).to(dtype)

    if c["op"] == "attn":
        b, s, h = c["batch"], c["s"], c["h"]
        lens = torch.randint(c["lmin"], c["lmax"] + 1, (b,), generator=gc)
        if b > 1 and c["lmin"] == 0:
            lens[0], lens[1] = 0, 1  # a padding entry of the batch, and a first token
        lens[-1] = c["lmax"]
        max_pages = -(-max(c["lmax"], 1) // PAGE)
        pages = b * max_pages
        kv = torch.empty(pages * PAGE, REC, dtype=torch.uint8, device=dev)
        for t in range(0, pages * PAGE, 1 << 18):
            kv[t:t + (1 << 18)] = _encode_fp4(randn(min(1 << 18, pages * PAGE - t), DIM))
        # Heads attend more or less sharply.
        q = (randn(b, s, h, DIM) * (0.5 + 2.5 * torch.rand(1, 1, h, 1, generator=g, device=dev))).to(torch.bfloat16)
        return dict(case=c, q=q, kv=kv.view(pages, PAGE, REC), lens=lens.to(torch.int32).to(dev),
                    table=torch.randperm(pages, generator=g, device=dev).to(torch.int32).view(b, max_pages),
                    out=torch.empty_like(q), lse=torch.empty(b, s, h, device=dev), longest=c["lmax"])
    if c["op"] == "norm":
        t = TYPES[c["dtype"]]
        n, d = c["n"], c["d"]
        x = randn(n, d) * torch.exp(randn(n, 1))
        x[:, :: max(1, d // 5)] *= 20.0  # a few channels carry outliers
        return dict(case=c, x=x.to(t), res=(3.0 * randn(n, d)).to(t) if c["residual"] else None,
                    w=(1.0 + 0.2 * randn(d)).to(t), codes=torch.empty(n, d, dtype=torch.uint8, device=dev),
                    scales=torch.empty(n, d // 32, dtype=torch.uint8, device=dev),
                    res_out=torch.empty(n, d, dtype=t, device=dev) if c["residual"] else None)
    if c["op"] == "rope":
        t = TYPES[c["dtype"]]
        x = randn(c["n"], c["h"], c["d"], dtype=t)
        return dict(case=c, x=x, out=x if c["inplace"] else torch.empty_like(x),
                    pos=torch.randint(0, c["maxpos"], (c["n"],), generator=g, device=dev, dtype=torch.int32))
    b = c["batch"]
    cached = torch.randint(0, c["cmax"] + 1, (b,), generator=gc)
    new = torch.randint(c["nmin"], c["nmax"] + 1, (b,), generator=gc)
    if c["gone"]:
        new[torch.randperm(b, generator=gc)[:c["gone"]]] = -1  # requests that have ended
    held = (cached + PAGE - 1) // PAGE
    # Room for the longest request and the fullest step, as a server's buffers have.
    max_pages = -(-(c["cmax"] + c["nmax"]) // PAGE)
    room = b * c["nmax"] + 7
    pages = b * max_pages + 100
    ids = torch.randperm(pages, generator=gc).to(torch.int32)
    table = torch.full((b, max_pages), -1, dtype=torch.int32)
    mine = torch.arange(max_pages).unsqueeze(0) < held.unsqueeze(1)
    table[mine] = ids[:int(held.sum())]
    free = torch.zeros(pages, dtype=torch.int32)
    spare = pages - int(held.sum())
    free[:spare] = ids[int(held.sum()):]
    i32 = lambda n: torch.empty(n, dtype=torch.int32, device=dev)  # noqa: E731
    return dict(case=c, cached=cached.to(torch.int32).to(dev), new=new.to(torch.int32).to(dev), table=table.to(dev),
                free=free.to(dev), num_free=torch.tensor([spare], dtype=torch.int32, device=dev),
                lens=i32(b), num_free_out=i32(1), cu=i32(b + 1), slots=i32(room), pos=i32(room))


# ---------------------------------------------------------------- one pass


def run(state):
    return {"attn": _attn, "norm": _norm, "rope": _rope, "plan": _plan}[state["case"]["op"]](state)


def _visible(c, lens, longest):
    """Positions [b, n] that some query token of a sequence may see (-1: none), and the mask [b, s, n]."""
    b, s, w, sinks = c["batch"], c["s"], c["window"], c["sinks"]
    end = lens.long().view(b, 1)
    if w == 0 or sinks + w + s - 1 >= longest:
        pos = torch.arange(max(longest, 1), device=lens.device).expand(b, -1)
    else:
        first = (end - s - w + 1).clamp_min(sinks)
        pos = torch.cat([torch.arange(sinks, device=lens.device).expand(b, -1),
                         first + torch.arange(w + s - 1, device=lens.device)], 1)
    at = (end - s + torch.arange(s, device=lens.device)).unsqueeze(2)  # [b, s, 1]: where each query token stands
    p = pos.unsqueeze(1)
    mask = p <= at
    if w:
        mask = mask & ((p > at - w) | (p < sinks))
    return pos, mask


def _attn(st):
    c = st["case"]
    if own:
        import fp4_kv_cache_sparse_gb300 as mla

        if "decoder" not in st:
            st["decoder"] = mla.PagedFP4Decoder(mla.PagedProblem.make(
                c["batch"], c["s"], c["h"], st["table"].shape[1], st["kv"].shape[0], window=c["window"],
                sinks=c["sinks"]))
        return st["decoder"](st["q"], st["kv"], st["table"], st["lens"], out=st["out"], lse=st["lse"])
    pos, mask = _visible(c, st["lens"], st["longest"])
    held = (pos < st["lens"].long().unsqueeze(1)) & (pos >= 0)
    where = torch.where(held, pos, 0)
    rec = st["kv"].view(-1, REC)[st["table"].long().gather(1, where // PAGE) * PAGE + where % PAGE]
    levels = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=rec.device)
    data = rec[..., :256]
    k = torch.stack([levels[(data & 15).int()], levels[(data >> 4).int()]], -1).flatten(-2)
    scale = rec[..., 256:].contiguous().view(torch.float8_e4m3fn).float()
    k = (k.unflatten(-1, (32, 16)) * scale.unsqueeze(-1)).flatten(-2)  # [b, n, 512]
    b, s, h = c["batch"], c["s"], c["h"]
    x = torch.matmul(st["q"].float().view(b, s * h, DIM), k.transpose(1, 2)).view(b, s, h, -1) / math.sqrt(DIM)
    x = x.masked_fill(~(mask & held.unsqueeze(1)).unsqueeze(2), -math.inf)
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(torch.isinf(m), 0.0, m))
    total = e.sum(-1, keepdim=True)
    o = torch.matmul((e / total.clamp_min(1e-30)).view(b, s * h, -1), k).view(b, s, h, DIM)
    return o.to(torch.bfloat16), (m + torch.log(total)).squeeze(-1)


def _norm(st):
    c = st["case"]
    if own:
        import fp4_kv_cache_sparse_gb300 as mla

        mla.rms_norm_fp8(st["x"], st["w"], 1e-6, st["codes"], st["scales"], residual=st["res"],
                         residual_out=st["res_out"])
        out = [st["codes"].view(torch.float8_e4m3fn), st["scales"].view(torch.float8_e8m0fnu)]
        return out + [st["res_out"]] if c["residual"] else out
    s = st["x"].float()
    if c["residual"]:
        s = s + st["res"].float()
    y = s * torch.rsqrt(s.square().mean(-1, keepdim=True) + 1e-6) * st["w"].float()
    y = y.view(c["n"], -1, 32)
    m, e = torch.frexp(y.abs().amax(-1))
    e = torch.where(m == 0, 0, torch.where(m <= 0.875, e - 9, e - 8)).clamp(-127, 127)
    codes = torch.ldexp(y, -e.unsqueeze(-1)).to(torch.float8_e4m3fn).view(c["n"], -1)
    scales = (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    return [codes, scales, s.to(st["x"].dtype)] if c["residual"] else [codes, scales]


def _frequencies(c, dev):
    """Radians per position of each pair, in 64 bits, and the factor on the result."""
    rd = c["rd"]
    j = torch.arange(rd // 2, dtype=torch.float64, device=dev)
    f = 10000.0 ** (-2.0 * j / rd)
    if c["scaling"] == "linear":
        return f / 8.0, 1.0
    if c["scaling"] == "yarn":
        turn = lambda r: rd * math.log(4096 / (r * 2 * math.pi)) / (2 * math.log(10000.0))  # noqa: E731
        low, high = max(math.floor(turn(32.0)), 0), min(math.ceil(turn(1.0)), rd - 1)
        ramp = ((j - low) / max(high - low, 0.001)).clamp(0, 1)
        return f * (1 - ramp) + f / 40.0 * ramp, 0.1 * math.log(40.0) + 1.0
    return f, 1.0


def _table(c):
    import fp4_kv_cache_sparse_gb300 as mla

    scaling = {"none": None, "linear": mla.RopeScaling.linear(8.0),
               "yarn": mla.RopeScaling.yarn(40.0, 4096)}[c["scaling"]]
    return mla.RopeTable(c["rd"], theta=10000.0, interleaved=c["layout"] == "interleaved", scaling=scaling,
                         attention_factor=1.0 if c["inplace"] else None)


def _rope(st):
    c, x = st["case"], st["x"]
    if own:
        import fp4_kv_cache_sparse_gb300 as mla

        if "rope" not in st:
            st["rope"] = _table(c)
        return mla.rope(x, st["pos"], st["rope"], offset=c["off"], out=st["out"])
    f, factor = _frequencies(c, x.device)
    factor = 1.0 if c["inplace"] else factor  # the same rows turn again and again: their length is kept
    phi = torch.remainder(st["pos"].double().unsqueeze(1) * f, 2 * math.pi).float().unsqueeze(1)
    cs, sn = torch.cos(phi) * factor, torch.sin(phi) * factor
    part = x[..., c["off"]:c["off"] + c["rd"]].float()
    if c["layout"] == "interleaved":
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([a * cs - b * sn, b * cs + a * sn], -1).flatten(-2)
    else:
        a, b = part.chunk(2, -1)
        turned = torch.cat([a * cs - b * sn, b * cs + a * sn], -1)
    if not c["inplace"]:
        st["out"].copy_(x)
    st["out"][..., c["off"]:c["off"] + c["rd"]] = turned.to(x.dtype)
    return st["out"]


def _plan(st):
    c = st["case"]
    if own:
        import fp4_kv_cache_sparse_gb300 as mla

        mla.page_plan(st["cached"], st["new"], st["table"], st["free"], st["num_free"], seq_lens=st["lens"],
                      num_free_out=st["num_free_out"], cu_new=st["cu"], slots=st["slots"], positions=st["pos"])
        return [st["lens"], st["num_free_out"], st["cu"], st["slots"], st["pos"], st["table"], st["free"]]
    cached, new, table, free = st["cached"].long(), st["new"].long(), st["table"], st["free"]
    gone, n = new < 0, new.clamp_min(0)
    held = (cached + PAGE - 1) // PAGE
    ends = torch.where(gone, 0, cached + n)
    zero = torch.zeros(1, dtype=torch.long, device=new.device)
    cu = torch.cat([zero, n.cumsum(0)])
    k = torch.arange(table.shape[1], device=new.device).unsqueeze(0)
    # Pages of ended requests go onto the stack, in order.
    back = gone.unsqueeze(1) & (k < held.unsqueeze(1))
    rank = torch.cumsum(back.flatten().long(), 0).view_as(back) - 1
    top = st["num_free"].long()
    last = free.numel()
    spare = torch.cat([free, free.new_zeros(1)])
    spare.scatter_(0, torch.where(back, top + rank, last).flatten(), torch.where(back, table, 0).flatten())
    free.copy_(spare[:last])
    top = top + back.sum()
    # New pages come from its top, in order.
    want = (k >= held.unsqueeze(1)) & (k < ((ends + PAGE - 1) // PAGE).unsqueeze(1)) & ~gone.unsqueeze(1)
    rank = torch.cumsum(want.flatten().long(), 0).view_as(want)
    table.copy_(torch.where(want, free[(top - rank).clamp(0, last - 1)], table))
    i = torch.arange(st["slots"].numel(), device=new.device)
    r = torch.searchsorted(cu[1:], i, right=True).clamp_max(c["batch"] - 1)
    live = i < cu[-1]
    pos = torch.where(live, cached[r] + i - cu[r], 0)
    page = table[r, (pos // PAGE).clamp_max(table.shape[1] - 1)]
    slots = torch.where(live, page * PAGE + pos % PAGE, -1)
    i32 = torch.int32
    return [ends.to(i32), (top - want.sum()).to(i32), cu.to(i32), slots.to(i32), pos.to(i32), table, free]


# ---------------------------------------------------------------- work and the definition in 64 bits


def work(case):
    c = case
    if c["op"] == "attn":
        per = (c["lmin"] + c["lmax"]) / 2.0
        seen = min(per, c["window"] + c["sinks"]) if c["window"] else per
        tokens = c["batch"] * max(seen, 1.0)
        rows = c["batch"] * c["s"] * c["h"]
        return {"bytes": tokens * REC + tokens / 16 + rows * (4 * DIM + 4), "flops": 4.0 * DIM * tokens * c["s"] * c["h"]}
    if c["op"] == "norm":
        e = 4 if c["dtype"] == "fp32" else 2
        return {"bytes": c["n"] * c["d"] * (e * (3 if c["residual"] else 1) + 1 + 1 / 32) + c["d"] * e,
                "flops": 8.0 * c["n"] * c["d"]}
    if c["op"] == "rope":
        e = 4 if c["dtype"] == "fp32" else 2
        return {"bytes": 2.0 * e * c["n"] * c["h"] * (c["rd"] if c["inplace"] else c["d"]) + 4 * c["n"],
                "flops": 3.0 * c["n"] * c["h"] * c["rd"]}
    tokens = c["batch"] * (c["nmin"] + c["nmax"]) / 2.0
    # Slots and positions are written to their end; a page is read and written for each that begins.
    return {"bytes": 8 * (c["batch"] * c["nmax"] + 7) + tokens / 8 + 16 * c["batch"], "flops": 0}


def exact(case, seed):
    st = prepare(case, seed)
    c, dev = case, torch.device("cuda")
    if c["op"] == "attn":
        levels = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device=dev)
        out = torch.zeros(c["batch"], c["s"], c["h"], DIM, dtype=torch.float64, device=dev)
        lse = torch.full((c["batch"], c["s"], c["h"]), -math.inf, dtype=torch.float64, device=dev)
        for b, n in enumerate(st["lens"].tolist()):
            if n == 0:
                continue
            rec = st["kv"][st["table"][b, : -(-n // PAGE)].long()].reshape(-1, REC)[:n]
            code = torch.stack([rec[:, :256] & 15, rec[:, :256] >> 4], 2).reshape(n, DIM).long()
            k = levels[code] * rec[:, 256:].contiguous().view(torch.float8_e4m3fn).double().repeat_interleave(16, 1)
            j = torch.arange(n, device=dev)
            for i in range(c["s"]):
                at = n - c["s"] + i
                see = j <= at
                if c["window"]:
                    see &= (j > at - c["window"]) | (j < c["sinks"])
                if not bool(see.any()):
                    continue
                ks = k[see]
                x = st["q"][b, i].double() @ ks.T * DIM ** -0.5
                lse[b, i] = torch.logsumexp(x, -1)
                out[b, i] = torch.softmax(x, -1) @ ks
        return out, lse
    if c["op"] == "norm":
        s = st["x"].double() + (st["res"].double() if c["residual"] else 0.0)
        y = s / torch.sqrt((s * s).sum(-1, keepdim=True) / c["d"] + 1e-6) * st["w"].double()
        y = y.reshape(c["n"], c["d"] // 32, 32)
        amax = y.abs().amax(-1)
        e = torch.ceil(torch.log2(amax / 448.0))
        e = torch.where(amax * torch.exp2(-e) > 448.0, e + 1, e)
        e = torch.where(amax * torch.exp2(1 - e) <= 448.0, e - 1, e)
        e = torch.where(amax == 0, 0.0, e.clamp(-127, 127))
        z = y * torch.exp2(-e).unsqueeze(-1)
        # e4m3: steps of 2^(floor(log2 z) - 3), 2^-9 below 2^-6.
        step = torch.exp2(torch.floor(torch.log2(z.abs().clamp_min(2.0 ** -6))) - 3)
        z = (torch.round(z / step) * step).reshape(c["n"], c["d"])
        return [z, torch.exp2(e), s] if c["residual"] else [z, torch.exp2(e)]
    if c["op"] == "rope":
        f, factor = _frequencies(c, dev)
        turn = torch.polar(torch.full_like(f, 1.0 if c["inplace"] else factor).expand(c["n"], -1).contiguous(),
                           st["pos"].double().outer(f)).unsqueeze(1)
        x = st["x"].double()
        part = x[..., c["off"]:c["off"] + c["rd"]]
        if c["layout"] == "interleaved":
            z = torch.view_as_real(torch.view_as_complex(part.reshape(c["n"], c["h"], -1, 2)) * turn).flatten(-2)
        else:
            z = torch.complex(part[..., : c["rd"] // 2].contiguous(), part[..., c["rd"] // 2:].contiguous()) * turn
            z = torch.cat([z.real, z.imag], -1)
        x[..., c["off"]:c["off"] + c["rd"]] = z
        return x
    return None
