"""What appending, page selection and shared prefixes are measured on.

Four operators around the pages of the 4-bit cache: records of new tokens with
their rotary positions applied on the way (kv_append), the means of full pages
in 8 bits (page_means), attention over the pages that those means select for
each query token (paged_sparse_decode_fp4), and attention for a batch whose
sequences share long prefixes (paged_shared_decode_fp4).  With `own` false `run`
computes them in plain torch operations; with `own` true it makes the calls that
a program makes of fp4_kv_cache_sparse_gb300.
"""
import math

import torch

own = False

PAGE = 64
DIM = 512
FP8, FP4 = 528, 288   # bytes of a record
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # One decode step of 64 requests: a token each, the tail of 64 dims turned.
        dict(name="append_64_fp4", op="append", n=64, rec=FP4, dtype="bf16", row=512, off=448, rd=64, layout="interleaved",
             scaling="none", maxpos=131072, spare=0),
        # A prefill chunk's latents as they lie in the projection's rows, long-context frequencies, some padding rows.
        dict(name="append_8191_fp4_strided", op="append", n=8191, rec=FP4, dtype="bf16", row=576, off=448, rd=64,
             layout="interleaved", scaling="yarn", maxpos=1048576, spare=57),
        # The latents of a whole long prompt in half precision into the 8-bit cache.
        dict(name="append_100000_fp8_fp16", op="append", n=100000, rec=FP8, dtype="fp16", row=512, off=0, rd=128, layout="half",
             scaling="linear", maxpos=131072, spare=0),
        # The pages that a prefill chunk completes.
        dict(name="means_8192", op="means", n=8192, dense=False),
        # Every page of a cache that was filled before: a list of its pages' last slots.
        dict(name="means_4096_pages", op="means", n=4096, dense=True),
        # One request, few heads: the latency of a single call.
        dict(name="sparse_b1_h16_l8k", op="sparse", batch=1, s=1, h=16, lmin=8000, lmax=8000, top=16, sinks=1, local=2),
        # An ordinary batch of decode steps over ragged long contexts.
        dict(name="sparse_b32_h64_l64k", op="sparse", batch=32, s=1, h=64, lmin=16384, lmax=65536, top=64, sinks=1, local=4),
        # Speculative decode (two tokens), all heads, 128k tokens: the means of 2048 pages a sequence are scored.
        dict(name="sparse_b32_s2_h128_l128k", op="sparse", batch=32, s=2, h=128, lmin=131000, lmax=131072, top=64, sinks=1,
             local=2),
        # Odd head count, three tokens, short and empty sequences, few pages.
        dict(name="sparse_b7_s3_h24_l5k", op="sparse", batch=7, s=3, h=24, lmin=0, lmax=5001, top=9, sinks=0, local=1),
        # Few requests after a common system prompt, few heads: latency.
        dict(name="shared_b8_h16_p4k", op="shared", batch=8, s=1, h=16, groups=1, pmin=4096, pmax=4096, omin=1, omax=200),
        # Many samples of one long prompt, all heads.
        dict(name="shared_b64_h128_p16k", op="shared", batch=64, s=1, h=128, groups=1, pmin=16384, pmax=16384, omin=64,
             omax=1024),
        # Three prompts, two tokens, an odd head count, ragged lengths and an empty sequence.
        dict(name="shared_b31_s2_h24_3p", op="shared", batch=31, s=2, h=24, groups=3, pmin=1, pmax=9001, omin=0, omax=700),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "means", "sparse", "sparse", "shared", "shared"])
    if op == "append":
        rd = 2 * rng.choice([16, 32, 32, 64, rng.randrange(1, 129)])
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        most = 100000 if dtype != "fp32" else 60000
        n = _log(rng, 1, most)
        return dict(op=op, n=n, rec=rng.choice([FP4, FP4, FP8]) if n < 50000 else FP8, dtype=dtype, row=rng.choice([512, 576, 640]),
                    off=rng.choice([0, 512 - rd]), rd=rd, layout=rng.choice(["interleaved", "half"]),
                    scaling=rng.choice(["none", "linear", "yarn"]), maxpos=_log(rng, 1000, 1 << 20), spare=rng.choice([0, n // 9]))
    if op == "means":
        dense = rng.random() < 0.3
        return dict(op=op, n=_log(rng, 1, 4096 if dense else 200000), dense=dense)
    if op == "sparse":
        h = rng.choice([16, 16, 32, 64, 128, rng.randrange(1, 129)])
        s = rng.choice([1, 1, 2, rng.randrange(1, 7)])
        batch = _log(rng, 1, 64)
        # No costlier than the largest listed cases, in means, in selected pages and in products.
        lmax = _log(rng, 200, min(131072, 32 * 131072 // batch))
        top = _log(rng, 4, max(4, min(256, 32 * 2 * 64 // (batch * s), 32 * 2 * 128 * 64 // (batch * s * h))))
        sinks = rng.choice([0, 1, 2])
        return dict(op=op, batch=batch, s=s, h=h, lmin=rng.choice([0, lmax // 2, lmax]), lmax=lmax, top=top, sinks=sinks,
                    local=rng.randrange(1, top - sinks + 1) if rng.random() < 0.3 else 1)
    h = rng.choice([16, 16, 32, 64, 128, rng.randrange(1, 129)])
    s = rng.choice([1, 1, 2, rng.randrange(1, 5)])
    batch = _log(rng, 1, 128)
    groups = rng.choice([1, 1, 2, rng.randrange(1, 9)])
    most = min(64 * 128 * 16384 // (batch * s * h), 65536, 64 * 16384 // batch)
    pmax = _log(rng, min(64, most), most)
    omax = _log(rng, 1, min(2048, 64 * 1024 // batch))
    return dict(op=op, batch=batch, s=s, h=h, groups=groups, pmin=pmax if groups == 1 else rng.choice([0, pmax // 2]), pmax=pmax,
                omin=rng.choice([0, omax]), omax=omax)


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


def _decode_fp4(rec, t=torch.float32):
    """uint8 [..., 288] -> the values [..., 512] that the records stand for, exactly."""
    levels = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=rec.device, dtype=t)
    data = rec[..., :256]
    k = torch.stack([levels[(data & 15).int()], levels[(data >> 4).int()]], -1).flatten(-2)
    scale = rec[..., 256:].contiguous().view(torch.float8_e4m3fn).to(t)
    return (k.unflatten(-1, (32, 16)) * scale.unsqueeze(-1)).flatten(-2)


def _pool(pages, g, dev):
    """Pages of records whose tokens have something in common, as a text's have."""
    kv = torch.empty(pages * PAGE, FP4, dtype=torch.uint8, device=dev)
    topics = torch.randn(pages, 1, DIM, generator=g, device=dev)
    step = 1 << 12
    for p in range(0, pages, step):
        m = min(step, pages - p)
        x = 0.6 * topics[p:p + m] + 0.8 * torch.randn(m, PAGE, DIM, generator=g, device=dev)
        kv[p * PAGE:(p + m) * PAGE] = _encode_fp4(x.view(m * PAGE, DIM))
    return kv.view(pages, PAGE, FP4), topics.view(pages, DIM)


def _means(kv):
    """The means of all pages as they are held: 8-bit codes [pages, 512] and the byte 127 + e of their scale [pages]."""
    codes, scales = [], []
    for part in kv.split(1 << 12):
        total = _decode_fp4(part, torch.float64).sum(1)
        amax = total.abs().amax(-1, keepdim=True)
        m, e = torch.frexp(amax)
        e = torch.where(amax == 0, 0, torch.where(m <= 127.0 / 128.0, e - 7, e - 6))
        codes.append(torch.round(total * torch.exp2(-e.double())).to(torch.int8))
        scales.append((torch.where(amax == 0, 0, e - 6) + 127).to(torch.uint8).squeeze(-1))
    return torch.cat(codes), torch.cat(scales)


def _mean_records(kv):
    codes, scales = _means(kv)
    rec = torch.zeros(kv.shape[0], 528, dtype=torch.uint8, device=kv.device)
    rec[:, :DIM] = codes.view(torch.uint8)
    rec[:, DIM] = scales
    return rec


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    gc = torch.Generator().manual_seed(seed)
    c = case

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    if c["op"] == "append":
        n = c["n"]
        x = randn(n, c["row"]) * torch.exp(0.5 * randn(n, 1))
        x[:, 3::101] *= 8.0  # a few channels carry outliers
        slots = torch.randperm(-(-n // PAGE) * PAGE, generator=g, device=dev)[:n].to(torch.int32)
        if c["spare"]:
            slots[-c["spare"]:] = -1  # rows of the padded batch
        pages = -(-n // PAGE)
        return dict(case=c, x=x.to(TYPES[c["dtype"]])[:, :DIM], slots=slots,
                    pos=torch.randint(0, c["maxpos"], (n,), generator=g, device=dev, dtype=torch.int32),
                    pool=torch.zeros(pages, PAGE, c["rec"], dtype=torch.uint8, device=dev))
    if c["op"] == "means":
        n = c["n"]
        pages = n if c["dense"] else -(-n // PAGE) + 3
        kv, _ = _pool(pages, g, dev)
        ids = torch.randperm(pages, generator=g, device=dev)
        i = torch.arange(n, device=dev)
        if c["dense"]:
            slots = ids * PAGE + PAGE - 1
        else:  # one request's tokens, the first page begun by an earlier chunk
            at = i + int(torch.randint(0, PAGE, (1,), generator=gc))
            slots = ids[at // PAGE] * PAGE + at % PAGE
        return dict(case=c, kv=kv, slots=slots.to(torch.int32), means=torch.zeros(pages, 528, dtype=torch.uint8, device=dev))
    b, s, h = c["batch"], c["s"], c["h"]
    sharp = 0.5 + 2.5 * torch.rand(1, 1, h, 1, generator=g, device=dev)  # heads attend more or less sharply
    if c["op"] == "sparse":
        lens = torch.randint(c["lmin"], c["lmax"] + 1, (b,), generator=gc)
        if b > 1 and c["lmin"] == 0:
            lens[0], lens[1] = 0, 1  # a padding entry of the batch, and a first token
        lens[-1] = c["lmax"]
        max_pages = -(-max(c["lmax"], 1) // PAGE)
        pages = b * max_pages
        kv, topics = _pool(pages, g, dev)
        table = torch.randperm(pages, generator=g, device=dev).view(b, max_pages)
        # Each head looks for what some page of its sequence is about.
        pick = (torch.rand(b, s, h, generator=g, device=dev) * (lens.to(dev).view(b, 1, 1) / PAGE)).long()
        want = topics[table.unsqueeze(1).expand(b, s, -1).gather(2, pick.clamp_max(max_pages - 1))]
        q = (0.9 * randn(b, s, h, DIM) + 0.4 * want) * sharp
        return dict(case=c, q=q.to(torch.bfloat16), kv=kv, means=_mean_records(kv), table=table.to(torch.int32),
                    lens=lens.to(torch.int32).to(dev), out=torch.empty(b, s, h, DIM, dtype=torch.bfloat16, device=dev),
                    lse=torch.empty(b, s, h, device=dev), sel=torch.empty(b, s, c["top"], dtype=torch.int32, device=dev))
    G = c["groups"]
    cuts = torch.sort(torch.randint(0, b + 1, (G - 1,), generator=gc)).values
    start = torch.cat([torch.zeros(1, dtype=torch.long), cuts, torch.tensor([b])])
    plens = torch.randint(c["pmin"], c["pmax"] + 1, (G,), generator=gc)
    plens[-1] = c["pmax"]
    lens = torch.randint(c["omin"], c["omax"] + 1, (b,), generator=gc)
    if b > 1 and c["omin"] == 0:
        lens[0] = 0  # a padding entry of the batch
    pp, op = -(-max(c["pmax"], 1) // PAGE), -(-max(c["omax"], 1) // PAGE)
    pages = G * pp + b * op
    kv, _ = _pool(pages, g, dev)
    ids = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    i32 = lambda v: v.to(torch.int32).to(dev)  # noqa: E731
    return dict(case=c, q=(randn(b, s, h, DIM) * sharp).to(torch.bfloat16), kv=kv, start=i32(start), plens=i32(plens),
                lens=i32(lens), ptable=ids[:G * pp].view(G, pp).contiguous(), table=ids[G * pp:].view(b, op).contiguous(),
                out=torch.empty(b, s, h, DIM, dtype=torch.bfloat16, device=dev), lse=torch.empty(b, s, h, device=dev))


# ---------------------------------------------------------------- one pass


def run(state):
    return {"append": _append, "means": _page_means, "sparse": _sparse, "shared": _shared}[state["case"]["op"]](state)


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


def _append(st):
    c, x = st["case"], st["x"]
    rec = st["pool"].view(-1, c["rec"])
    if own:
        import fp4_kv_cache_sparse_gb300 as mla

        if "rope" not in st:
            scaling = {"none": None, "linear": mla.RopeScaling.linear(8.0),
                       "yarn": mla.RopeScaling.yarn(40.0, 4096)}[c["scaling"]]
            st["rope"] = mla.RopeTable(c["rd"], theta=10000.0, interleaved=c["layout"] == "interleaved", scaling=scaling)
        kind = mla.KV_FP8_528 if c["rec"] == FP8 else mla.KV_FP4_288
        mla.kv_append(x, st["slots"], st["pool"], kind, rope=st["rope"], positions=st["pos"], offset=c["off"])
        if c["rec"] == FP8:
            return [rec[:, :DIM].view(torch.float8_e4m3fn), rec[:, DIM:].view(torch.float8_e8m0fnu)]
        return mla.dequantize(rec, mla.KV_FP4_288)  # two values share a byte: the records as what they stand for
    f, factor = _frequencies(c, x.device)
    phi = torch.remainder(st["pos"].double().unsqueeze(1) * f, 2 * math.pi).float()
    cs, sn = torch.cos(phi) * factor, torch.sin(phi) * factor
    y = x.float()
    part = y[:, c["off"]:c["off"] + c["rd"]]
    if c["layout"] == "interleaved":
        a, b = part[:, 0::2], part[:, 1::2]
        turned = torch.stack([a * cs - b * sn, b * cs + a * sn], -1).flatten(-2)
    else:
        a, b = part.chunk(2, -1)
        turned = torch.cat([a * cs - b * sn, b * cs + a * sn], -1)
    y = torch.cat([y[:, :c["off"]], turned, y[:, c["off"] + c["rd"]:]], 1)
    live = st["slots"] >= 0
    slots = st["slots"].long()[live]
    y = y[live]
    if c["rec"] == FP8:
        y = y.view(-1, 16, 32)
        m, e = torch.frexp(y.abs().amax(-1))
        e = torch.where(m == 0, 0, torch.where(m <= 0.875, e - 9, e - 8)).clamp(-127, 127)
        rec[slots, :DIM] = torch.ldexp(y, -e.unsqueeze(-1)).to(torch.float8_e4m3fn).view(torch.uint8).view(-1, DIM)
        rec[slots, DIM:] = (e + 127).to(torch.uint8)
        return [rec[:, :DIM].view(torch.float8_e4m3fn), rec[:, DIM:].view(torch.float8_e8m0fnu)]
    y = y.view(-1, 32, 16)
    sc = (y.abs().amax(-1) / 6.0).clamp_max(448.0).to(torch.float8_e4m3fn)
    t = torch.where(sc.float().unsqueeze(-1) == 0, 0.0, y / sc.float().unsqueeze(-1))
    # The nearest level; halfway between two the one with the even code.
    down = torch.tensor([0.25, 1.25, 2.5, 5.0], device=x.device)
    up = torch.tensor([0.75, 1.75, 3.5], device=x.device)
    code = torch.bucketize(t.abs(), down) + torch.bucketize(t.abs(), up, right=True)
    code = (code.to(torch.uint8) | (torch.signbit(t).to(torch.uint8) << 3)).view(-1, 256, 2)
    rec[slots, :256] = code[..., 0] | (code[..., 1] << 4)
    rec[slots, 256:] = sc.view(torch.uint8)
    return _decode_fp4(rec).to(torch.bfloat16)


def _page_means(st):
    means = st["means"]
    if own:
        import fp4_kv_cache_sparse_gb300 as mla

        mla.page_means(st["kv"], st["slots"], means)
    else:
        slots = st["slots"].long()
        pages = (slots // PAGE)[slots % PAGE == PAGE - 1]
        codes, scales = _means(st["kv"][pages])
        means[pages, :DIM] = codes.view(torch.uint8)
        means[pages, DIM] = scales
    return [means[:, :DIM].view(torch.int8), means[:, DIM:DIM + 1].view(torch.float8_e8m0fnu)]


def _softmax_over(q, k, see):
    """q [b, r, 512], k [b, n, 512] in 32 bits, see [b, r, n]: outputs and log-sum-exps; rows that see nothing give 0 and -inf."""
    x = (torch.matmul(q, k.transpose(1, 2)) / math.sqrt(DIM)).masked_fill(~see, -math.inf)
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(torch.isinf(m), 0.0, m))
    total = e.sum(-1, keepdim=True)
    return torch.matmul(e / total.clamp_min(1e-30), k), (m + torch.log(total)).squeeze(-1)


def _select(c, q, codes, scales, table, at):
    """The pages [b, s, top] that each query token attends to, in order, -1 after the last; `at` [b, s] is where it stands."""
    b, s, h, top = c["batch"], c["s"], c["h"], c["top"]
    amax = q.abs().amax(-1)
    m, e = torch.frexp(amax)
    e = torch.where(m <= 127.0 / 128.0, e - 7, e - 6).clamp_min(-120)
    a = torch.round(q * torch.exp2(-e.float()).unsqueeze(-1))
    e = torch.where(amax == 0, -1000, e)
    weight = torch.exp2((e - e.amax(-1, keepdim=True)).clamp_min(-100).float())  # [b, s, h]
    # Integers below 2^24 in magnitude: exact in 32 bits, whatever the order.
    dots = torch.matmul(a.view(b, s * h, DIM), codes[table].float().transpose(1, 2)).view(b, s, h, -1)
    score = (dots * weight.unsqueeze(-1)).amax(2) * torch.exp2(scales[table].float() - 127.0).unsqueeze(1)
    j = torch.arange(table.shape[1], device=q.device)
    mine = torch.where(at >= 0, at // PAGE, -1).unsqueeze(-1)  # [b, s, 1]
    held = j <= mine
    always = held & ((j < c["sinks"]) | (j > mine - c["local"]))
    left = top - always.sum(-1, keepdim=True)
    score = score.masked_fill(~held | always, -math.inf)
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(2, order, j.expand_as(order))
    chosen = always | (held & ~always & (rank < left))
    pages = torch.where(chosen, j, 1 << 30)
    pages = torch.nn.functional.pad(pages, (0, max(0, top - pages.shape[-1])), value=1 << 30)
    pages = torch.sort(pages, dim=-1).values[..., :top]
    return torch.where(pages < (1 << 30), pages, -1)


def _sparse(st):
    c = st["case"]
    b, s, h, top = c["batch"], c["s"], c["h"], c["top"]
    if own:
        import fp4_kv_cache_sparse_gb300 as mla

        if "decoder" not in st:
            st["decoder"] = mla.PagedSparseFP4Decoder(mla.PagedSparseProblem.make(
                b, s, h, st["table"].shape[1], st["kv"].shape[0], top, sink_pages=c["sinks"], local_pages=c["local"]))
        return st["decoder"](st["q"], st["kv"], st["means"], st["table"], st["lens"], out=st["out"], lse=st["lse"],
                             selected=st["sel"])
    table, lens, q = st["table"].long(), st["lens"].long(), st["q"].float()
    at = lens.view(b, 1) - s + torch.arange(s, device=q.device)  # where each query token stands
    sel = _select(c, q, st["means"][:, :DIM].view(torch.int8), st["means"][:, DIM], table, at)
    rows = table.unsqueeze(1).expand(b, s, -1).gather(2, sel.clamp_min(0))
    k = _decode_fp4(st["kv"][rows]).view(b * s, top * PAGE, DIM)
    pos = (sel.unsqueeze(-1) * PAGE + torch.arange(PAGE, device=q.device)).view(b, s, 1, -1)
    see = (sel >= 0).repeat_interleave(PAGE, -1).unsqueeze(2) & (pos <= at.view(b, s, 1, 1))
    out, lse = _softmax_over(q.view(b * s, h, DIM), k, see.view(b * s, 1, -1))
    return out.view(b, s, h, DIM).to(torch.bfloat16), lse.view(b, s, h), sel.to(torch.int32)


def _shared(st):
    c = st["case"]
    b, s, h, G = c["batch"], c["s"], c["h"], c["groups"]
    if own:
        import fp4_kv_cache_sparse_gb300 as mla

        if "decoder" not in st:
            st["decoder"] = mla.PagedSharedFP4Decoder(mla.PagedSharedProblem.make(
                b, s, h, st["table"].shape[1], st["ptable"].shape[1], st["kv"].shape[0], groups=G))
        return st["decoder"](st["q"], st["kv"], st["start"], st["ptable"], st["plens"], st["table"], st["lens"],
                             out=st["out"], lse=st["lse"])
    dev = st["q"].device
    q = st["q"].float().view(b, s * h, DIM)
    mine = _decode_fp4(st["kv"][st["table"].long()]).view(b, -1, DIM)
    pre = _decode_fp4(st["kv"][st["ptable"].long()]).view(G, -1, DIM)
    at = (st["lens"].long().view(b, 1) - s + torch.arange(s, device=dev)).repeat_interleave(h, 1).unsqueeze(-1)
    see_mine = torch.arange(mine.shape[1], device=dev) <= at
    group = (torch.searchsorted(st["start"].long(), torch.arange(b, device=dev), right=True) - 1).clamp(0, G - 1)
    see_pre = (torch.arange(pre.shape[1], device=dev) < st["plens"].long()[group].view(b, 1, 1)) & (at >= 0)
    if G == 1:  # one product for the whole batch
        x = torch.matmul(q.view(1, -1, DIM), pre.transpose(1, 2)).view(b, s * h, -1)
    else:
        x = torch.matmul(q, pre[group].transpose(1, 2))
    x = (x / math.sqrt(DIM)).masked_fill(~see_pre, -math.inf)
    y = (torch.matmul(q, mine.transpose(1, 2)) / math.sqrt(DIM)).masked_fill(~see_mine, -math.inf)
    m = torch.maximum(x.amax(-1, keepdim=True), y.amax(-1, keepdim=True))
    base = torch.where(torch.isinf(m), 0.0, m)
    x, y = torch.exp(x - base), torch.exp(y - base)
    total = x.sum(-1, keepdim=True) + y.sum(-1, keepdim=True)
    if G == 1:
        o = torch.matmul(x.view(1, b * s * h, -1), pre).view(b, s * h, DIM)
    else:
        o = torch.matmul(x, pre[group])
    o = (o + torch.matmul(y, mine)) / total.clamp_min(1e-30)
    return o.view(b, s, h, DIM).to(torch.bfloat16), (m + torch.log(total)).view(b, s, h)


# ---------------------------------------------------------------- work and the definition in 64 bits


def work(case):
    c = case
    if c["op"] == "append":
        e = 4 if c["dtype"] == "fp32" else 2
        read_back = 0 if c["rec"] == FP8 else FP4 + 2 * DIM  # 4-bit records are read back as values
        return {"bytes": c["n"] * (DIM * e + 8 + c["rec"] + read_back), "flops": 3.0 * c["n"] * c["rd"]}
    if c["op"] == "means":
        pages = c["n"] if c["dense"] else max(1, c["n"] // PAGE)
        return {"bytes": 4 * c["n"] + pages * (PAGE * FP4 + DIM + 1), "flops": 2.0 * pages * PAGE * DIM}
    if c["op"] == "sparse":
        pages = max((c["lmin"] + c["lmax"]) / 2.0 / PAGE, 1.0)
        queries = c["batch"] * c["s"]
        top = min(c["top"], pages)
        return {"bytes": c["batch"] * pages * (DIM + 5) + min(queries * top, c["batch"] * pages) * PAGE * FP4
                + queries * (c["h"] * (4 * DIM + 4) + 4 * c["top"]),
                "flops": queries * c["h"] * DIM * (2.0 * pages + 4.0 * PAGE * top)}
    prefix = c["groups"] * (c["pmin"] + c["pmax"]) / 2.0
    mine = c["batch"] * (c["omin"] + c["omax"]) / 2.0
    rows = c["batch"] * c["s"] * c["h"]
    return {"bytes": (prefix + mine) * (FP4 + 1 / 16) + rows * (4 * DIM + 4),
            "flops": 4.0 * DIM * rows * (prefix / c["groups"] + mine / c["batch"])}


def exact(case, seed):
    st = prepare(case, seed)
    c, dev = case, torch.device("cuda")
    if c["op"] == "append":
        f, factor = _frequencies(c, dev)
        turn = torch.polar(torch.full_like(f, factor).expand(c["n"], -1).contiguous(), st["pos"].double().outer(f))
        y = st["x"].double()
        part = y[:, c["off"]:c["off"] + c["rd"]]
        if c["layout"] == "interleaved":
            z = torch.view_as_real(torch.view_as_complex(part.reshape(c["n"], -1, 2)) * turn).flatten(-2)
        else:
            z = torch.complex(part[:, :c["rd"] // 2].contiguous(), part[:, c["rd"] // 2:].contiguous()) * turn
            z = torch.cat([z.real, z.imag], -1)
        y[:, c["off"]:c["off"] + c["rd"]] = z
        live = st["slots"] >= 0
        slots, y = st["slots"].long()[live], y[live]
        total = st["pool"].numel() // c["rec"]

        def e4m3(v):  # steps of 2^(floor(log2 v) - 3), 2^-9 below 2^-6, 448 at most
            step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
            return (torch.round(v / step) * step).clamp(-448.0, 448.0)

        if c["rec"] == FP8:
            y = y.view(-1, 16, 32)
            amax = y.abs().amax(-1)
            e = torch.ceil(torch.log2(amax / 448.0))
            e = torch.where(amax * torch.exp2(-e) > 448.0, e + 1, e)
            e = torch.where(amax * torch.exp2(1 - e) <= 448.0, e - 1, e)
            e = torch.where(amax == 0, 0.0, e.clamp(-127, 127))
            codes = torch.zeros(total, DIM, dtype=torch.float64, device=dev)
            scales = torch.full((total, 16), 2.0 ** -127, dtype=torch.float64, device=dev)
            codes[slots] = e4m3(y * torch.exp2(-e).unsqueeze(-1)).view(-1, DIM)
            scales[slots] = torch.exp2(e)
            return [codes, scales]
        y = y.view(-1, 32, 16)
        sc = e4m3(y.abs().amax(-1) / 6.0).unsqueeze(-1)
        t = torch.where(sc == 0, 0.0, y / sc).clamp(-6.0, 6.0)
        step = torch.exp2(torch.floor(torch.log2(t.abs().clamp_min(1.0))) - 1)  # e2m1: halves up to 2, then 1, then 2
        values = torch.zeros(total, DIM, dtype=torch.float64, device=dev)
        values[slots] = (torch.round(t / step) * step * sc).view(-1, DIM)
        return values
    if c["op"] == "means":
        codes = torch.zeros(st["kv"].shape[0], DIM, dtype=torch.int8, device=dev)
        scales = torch.full((st["kv"].shape[0], 1), 2.0 ** -127, dtype=torch.float64, device=dev)
        slots = st["slots"].long()
        for page in (slots[slots % PAGE == PAGE - 1] // PAGE).split(1 << 10):
            mean = _decode_fp4(st["kv"][page], torch.float64).mean(1)
            amax = mean.abs().amax(-1, keepdim=True)
            e = torch.ceil(torch.log2(amax / 127.0))
            e = torch.where(amax * torch.exp2(-e) > 127.0, e + 1, e)
            e = torch.where(amax * torch.exp2(1 - e) <= 127.0, e - 1, e)
            e = torch.where(amax == 0, 0.0, e)
            codes[page] = torch.round(mean / torch.exp2(e)).to(torch.int8)
            scales[page] = torch.where(amax == 0, 1.0, torch.exp2(e))
        return [codes, scales]
    b, s, h = c["batch"], c["s"], c["h"]
    out = torch.zeros(b, s, h, DIM, dtype=torch.float64, device=dev)
    lse = torch.full((b, s, h), -math.inf, dtype=torch.float64, device=dev)
    if c["op"] == "sparse":
        sel = torch.full((b, s, c["top"]), -1, dtype=torch.int32, device=dev)
        codes = st["means"][:, :DIM].view(torch.int8)
        for r, n in enumerate(st["lens"].tolist()):
            ids = st["table"][r].long()
            mean = codes[ids].double() * torch.exp2(st["means"][ids, DIM].double() - 127).unsqueeze(1)
            for i in range(s):
                at = n - s + i
                if at < 0:
                    continue
                q = st["q"][r, i].double()
                amax = q.abs().amax(-1, keepdim=True)
                e = torch.ceil(torch.log2(amax / 127.0))
                e = torch.where(amax * torch.exp2(-e) > 127.0, e + 1, e)
                e = torch.where(amax * torch.exp2(1 - e) <= 127.0, e - 1, e)
                e = torch.where(amax == 0, 0.0, e)
                score = (torch.round(q / torch.exp2(e)) * torch.exp2(e) @ mean.T).amax(0)
                last = at // PAGE
                keep = [j for j in range(last + 1) if j < c["sinks"] or j > last - c["local"]]
                rest = [j for j in range(last + 1) if c["sinks"] <= j <= last - c["local"]]
                v = score.tolist()
                pages = sorted(keep + sorted(rest, key=lambda j: (-v[j], j))[:max(0, c["top"] - len(keep))])
                sel[r, i, :len(pages)] = torch.tensor(pages, dtype=torch.int32, device=dev)
                k = _decode_fp4(st["kv"][ids[torch.tensor(pages, device=dev)]], torch.float64).view(-1, DIM)
                k = k[:(len(pages) - 1) * PAGE + at % PAGE + 1]
                x = q @ k.T * DIM ** -0.5
                lse[r, i], out[r, i] = torch.logsumexp(x, -1), torch.softmax(x, -1) @ k
        return out, lse, sel
    start = st["start"].tolist()
    for g in range(c["groups"]):
        n = int(st["plens"][g])
        pre = _decode_fp4(st["kv"][st["ptable"][g, :-(-n // PAGE)].long()], torch.float64).view(-1, DIM)[:n]
        for r in range(start[g], start[g + 1]):
            m = int(st["lens"][r])
            k = torch.cat([pre, _decode_fp4(st["kv"][st["table"][r, :-(-m // PAGE)].long()], torch.float64).view(-1, DIM)[:m]])
            for i in range(s):
                see = n + m - s + i + 1 if m - s + i >= 0 else 0
                if see:
                    x = st["q"][r, i].double() @ k[:see].T * DIM ** -0.5
                    lse[r, i], out[r, i] = torch.logsumexp(x, -1), torch.softmax(x, -1) @ k[:see]
    return out, lse
