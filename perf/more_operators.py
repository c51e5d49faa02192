"""The operators of a decode step around the latent cache, as measured cases.

  rope      rotary positions of a batch's queries: interleaved and half layouts, the rotary part of wider heads,
            frequencies scaled for long contexts (mla_rope).
  append    from a projection's output to cached rows: the latent's norm, the rotation of the shared key, and the
            write into each request's pages, as bf16, 656-byte or page-scaled 8-bit rows (mla_cache_append).
  decode    attention over 8-bit rows with one scale for each page of tokens (mla_decode_fp8_page).

A case names an operator and its sizes. The lengths of its requests are drawn from the case's own "lens" number, so
they are part of the case; the values are drawn from the seed.
"""
import math

import numpy as np
import torch

own = False

SCALE = 1.0 / math.sqrt(192.0)
EPS = 1e-6
ROW_BYTES = {"bf16": 1152, "fp8": 656, "page8": 576}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one step of 64 requests deep in long contexts: the rotary part of 192-wide query heads, into the decode's own buffer
        {"name": "rope_step", "op": "rope", "dtype": "bf16", "T": 64, "H": 16, "R": 64, "width": 192, "layout": "interleaved",
         "scaling": "yarn", "far": 160000, "packed_out": True},
        # the queries of a whole prompt behind a million tokens
        {"name": "rope_prompt", "op": "rope", "dtype": "bf16", "T": 32768, "H": 16, "R": 64, "width": 192,
         "layout": "interleaved", "scaling": "yarn", "far": 1000000, "packed_out": False},
        # the gradient's way back through the rotation, in 32 bits, an odd number of tokens, half layout
        {"name": "rope_back_f32", "op": "rope", "dtype": "f32", "T": 4099, "H": 20, "R": 64, "width": 64, "layout": "half",
         "scaling": "linear", "far": 30000, "packed_out": True, "back": True},
        # one token for each of 64 requests, 8-bit rows: what a step pays in every layer
        {"name": "append_step", "op": "append", "kind": "page8", "B": 64, "n_lo": 1, "n_hi": 1, "p_lo": 1000, "p_hi": 8192,
         "page": 64, "norm": True, "layout": "interleaved", "scaling": "yarn", "dense": False, "given": False, "lens": 1},
        # a verify step of four tokens, bf16 rows, positions that earlier evictions left behind the places
        {"name": "append_verify", "op": "append", "kind": "bf16", "B": 128, "n_lo": 4, "n_hi": 4, "p_lo": 0, "p_hi": 4000,
         "page": 16, "norm": True, "layout": "half", "scaling": "none", "dense": False, "given": True, "lens": 2},
        # a batch of ragged prompts into 8-bit pages, with the dense rows that the up-projection reads
        {"name": "append_prompts", "op": "append", "kind": "page8", "B": 16, "n_lo": 1, "n_hi": 8192, "p_lo": 0, "p_hi": 300,
         "page": 64, "norm": True, "layout": "interleaved", "scaling": "yarn", "dense": True, "given": False, "lens": 3},
        # one long document into 656-byte rows
        {"name": "append_long_fp8", "op": "append", "kind": "fp8", "B": 1, "n_lo": 98304, "n_hi": 98304, "p_lo": 0, "p_hi": 0,
         "page": 64, "norm": True, "layout": "interleaved", "scaling": "yarn", "dense": False, "given": False, "lens": 4},
        # two requests: what a call costs before any work
        {"name": "decode_tiny", "op": "decode", "B": 2, "t_lo": 37, "t_hi": 200, "Hq": 8, "q_len": 1, "page": 16, "lens": 5},
        # a serving batch at 16 heads
        {"name": "decode_batched", "op": "decode", "B": 64, "t_lo": 1024, "t_hi": 8192, "Hq": 16, "q_len": 1, "page": 16,
         "lens": 6},
        # few very long contexts
        {"name": "decode_long", "op": "decode", "B": 4, "t_lo": 262144, "t_hi": 262144, "Hq": 32, "q_len": 1, "page": 64,
         "lens": 7},
        # 64 query rows
        {"name": "decode_wide", "op": "decode", "B": 32, "t_lo": 16384, "t_hi": 32768, "Hq": 64, "q_len": 1, "page": 64,
         "lens": 8},
        # a verify step of eight tokens at 16 heads: 128 query rows
        {"name": "decode_verify", "op": "decode", "B": 32, "t_lo": 1, "t_hi": 24000, "Hq": 16, "q_len": 8, "page": 32,
         "lens": 9},
    ]


def draw(rng):
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    op = rng.choice(("rope", "append", "decode"))
    layout, scaling = rng.choice(("half", "interleaved")), rng.choice(("none", "linear", "yarn"))
    if op == "rope":
        H, R = rng.choice((1, 8, 16, 20, 32, 64, 128)), rng.choice((64, 64, 64, 32, 128, 24))
        return {"op": op, "dtype": rng.choice(("bf16", "f32")), "T": log(1, (1 << 24) // (H * R)), "H": H, "R": R,
                "width": R + rng.choice((0, 8, 128)), "layout": layout, "scaling": scaling, "far": log(1, 1000000),
                "packed_out": rng.random() < 0.5, "back": rng.random() < 0.3}
    case = {"op": op, "lens": rng.randrange(1 << 30), "page": rng.choice((1, 3, 8, 16, 16, 64, 64, 96))}
    if op == "append":
        B = log(1, 160)
        hi = log(1, 90000 // B)
        case.update(kind=rng.choice(("bf16", "fp8", "page8", "page8")), B=B, n_lo=rng.randint(0, hi), n_hi=hi,
                    p_lo=0, p_hi=log(1, max(1, min(9000, 400000 // B))), norm=rng.random() < 0.8, layout=layout, scaling=scaling,
                    dense=rng.random() < 0.4, given=rng.random() < 0.3)
        return case
    B = log(1, 96)
    Hq, q_len = rng.choice(((1, 1), (8, 1), (16, 1), (20, 1), (32, 1), (64, 1), (128, 1), (16, 2), (16, 4), (8, 7), (16, 8)))
    hi = log(2, min(262144, 1000000 // B, 48000000 // (B * Hq * q_len)))
    case.update(B=B, t_lo=rng.randint(0, hi), t_hi=hi, Hq=Hq, q_len=q_len)
    return case


def _draw_lens(case, lo, hi):
    r = np.random.default_rng(case["lens"])
    n = r.integers(lo, hi, size=case["B"], endpoint=True)
    n[0] = hi
    return n, r


def _tokens(case):
    """append: new tokens and tokens before them, by request; decode: cached tokens."""
    if case["op"] == "decode":
        return _draw_lens(case, case["t_lo"], case["t_hi"])[0]
    n, r = _draw_lens(case, case["n_lo"], case["n_hi"])
    return n, r.integers(case["p_lo"], case["p_hi"], size=case["B"], endpoint=True)


def work(case):
    if case["op"] == "rope":
        n = case["T"] * case["H"] * case["R"]
        return {"bytes": n * 2 * (2 if case["dtype"] == "bf16" else 4) + case["T"] * 4, "flops": 3 * n}
    if case["op"] == "append":
        n, before = _tokens(case)
        tok, page = int(n.sum()), case["page"]
        touched = int(np.where(n > 0, (before + n - 1) // page - before // page + 1, 0).sum())
        return {"bytes": tok * (1152 + ROW_BYTES[case["kind"]] + (1152 if case["dense"] else 0)) +
                (4 * touched if case["kind"] == "page8" else 0), "flops": 5 * 576 * tok}
    t, rows = _tokens(case), case["Hq"] * case["q_len"]
    n = int(t.sum())
    return {"bytes": n * 576 + 4 * int((-(-t // case["page"])).sum()) + case["B"] * rows * (1152 + 1024 + 4),
            "flops": 2 * (576 + 512) * rows * n}


# --------------------------------------------------------------- the inputs

def _frequencies(R, scaling):
    """Radians a position turns each pair by (64 bits), and the factor on the rotated values.

    linear: positions shrunk by 4. yarn: by 40 where a pair turns less than once in 4096 positions, not at all
    where it turns more than 32 times, a ramp between the two, values times 0.1 ln 40 + 1."""
    i = np.arange(R // 2, dtype=np.float64)
    f = 10000.0 ** (-2.0 * i / R)
    if scaling == "linear":
        return f / 4.0, 1.0
    if scaling == "yarn":
        dim = lambda turns: R * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(10000.0))  # noqa: E731
        lo, hi = max(math.floor(dim(32)), 0), min(math.ceil(dim(1)), R - 1)
        ramp = np.clip((i - lo) / max(hi - lo, 0.001), 0.0, 1.0)
        return f / 40.0 * ramp + f * (1.0 - ramp), 0.1 * math.log(40.0) + 1.0
    return f, 1.0


def _steps(f):
    """The same as fractions of a turn in 64 bits, which a position multiplies modulo a turn."""
    turns = [int(x / (2 * math.pi) * 2.0 ** 64) for x in f.tolist()]
    return torch.tensor([t - (1 << 64) if t >= 1 << 63 else t for t in turns], dtype=torch.int64, device="cuda")


def _pages(t, page, gen):
    """Shuffled pages: the table [B, most] (-1 past a request's last page) and the pool's pages."""
    need = -(-t // page)
    ids = torch.randperm(max(1, int(need.sum() * 5 // 4)), generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(t), max(1, int(need.max()))), -1, dtype=torch.int32, device="cuda")
    cols = torch.arange(table.shape[1], device="cuda")[None] < torch.from_numpy(need).cuda()[:, None]
    table[cols] = ids[:int(need.sum())]
    return table, ids.numel()


def _pow2(top):
    """The least power of two s with top <= 448 s, within 2^-40 .. 2^40."""
    m, e = torch.frexp(top)
    e = torch.where(top > 0, torch.where(m > 0.875, e - 8, e - 9), -40).clamp(-40, 40)
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)  # the power itself, exactly


def _pool(kind, pages, page, gen):
    """Rows as earlier steps left them: N(0,1) latents and rotary keys."""
    slots = pages * page
    pool = torch.empty((slots, ROW_BYTES[kind]), dtype=torch.uint8, device="cuda")
    scales = torch.ones((pages,), dtype=torch.float32, device="cuda")
    step = max(1, (1 << 18) // page)
    for a in range(0, pages, step):
        n = min(step, pages - a)
        at = slice(a * page, (a + n) * page)
        x = torch.randn((n * page, 576), generator=gen, device="cuda").to(torch.bfloat16)
        if kind == "bf16":
            pool[at] = x.view(torch.uint8)
        elif kind == "fp8":
            v = x[:, :512].float().view(-1, 4, 128)
            s = v.abs().amax(2) / 448.0
            pool[at, :512] = (v / s[:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(-1, 512)
            pool[at, 512:528] = s.view(torch.uint8)
            pool[at, 528:] = x[:, 512:].contiguous().view(torch.uint8)
        else:
            # pages of different loudness, as layers and documents have them
            loud = torch.exp(0.5 * torch.randn((n, 1), generator=gen, device="cuda"))
            v = x.float().view(n, page * 576) * loud
            s = _pow2(v.abs().amax(1))
            pool[at] = (v / s[:, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(-1, 576)
            scales[a:a + n] = s
    return pool, scales


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": dict(case)}
    i32 = lambda x: torch.from_numpy(np.asarray(x, dtype=np.int32)).cuda()  # noqa: E731
    randn = lambda *n: torch.randn(n, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    if case["op"] != "decode":
        f, s["mscale"] = _frequencies(case.get("R", 64), case["scaling"])
        s.update(freq=torch.from_numpy(f).cuda(), steps=_steps(f))
    if case["op"] == "rope":
        T, H, R, width = case["T"], case["H"], case["R"], case["width"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        if case.get("back"):
            s.update(freq=-s["freq"], steps=-s["steps"])
        heads = torch.randn((T, H, width), generator=gen, device="cuda").to(dt)
        out = torch.zeros((T, H, R if case["packed_out"] else width), dtype=dt, device="cuda")
        s.update(x=heads[:, :, width - R:], out=out[:, :, out.shape[2] - R:],
                 pos=case["far"] + torch.randint(0, 4096, (T,), generator=gen, device="cuda", dtype=torch.int32))
        return s
    if case["op"] == "append":
        n, before = _tokens(case)
        tok = int(n.sum())
        table, pages = _pages(n + before, case["page"], gen)
        pool, scales = _pool(case["kind"], pages, case["page"], gen)
        # one projection's output: latent and rotary key side by side, some tokens louder than others
        proj = (torch.randn((tok, 576), generator=gen, device="cuda") *
                torch.exp(0.5 * torch.randn((tok, 1), generator=gen, device="cuda"))).to(torch.bfloat16)
        s.update(latent=proj[:, :512], k_pe=proj[:, 512:], cu=i32(np.concatenate([[0], np.cumsum(n)])), lens=i32(n + before),
                 table=table, cache=pool, scales=scales, total=tok, w=(1 + 0.1 * randn(512).float()).to(torch.bfloat16) if case["norm"] else None,
                 rows=torch.zeros((tok, 576), dtype=torch.bfloat16, device="cuda") if case["dense"] else None, pos=None)
        if case["given"]:
            place = np.concatenate([np.arange(b, b + m) + 1000 + 7 * k for k, (m, b) in enumerate(zip(n.tolist(), before.tolist()))])
            s["pos"] = i32(place)
        return s
    t = _tokens(case)
    table, pages = _pages(t, case["page"], gen)
    rows = case["B"] * case["q_len"]
    s["cache"], s["scales"] = _pool("page8", pages, case["page"], gen)
    s.update(table=table, lens=i32(t), most=max(1, int(t.max())), q_lat=randn(rows, case["Hq"], 512), q_pe=randn(rows, case["Hq"], 64),
             out=torch.zeros((rows, case["Hq"], 512), dtype=torch.bfloat16, device="cuda"),
             lse=torch.zeros((rows, case["Hq"]), dtype=torch.float32, device="cuda"), workspace=None)
    # room for any device's partial results, kept from step to step
    groups = -(-case["Hq"] * case["q_len"] // 64)
    s["workspace"] = torch.empty((1 << 20) + groups * (160 + case["B"]) * 64 * (513 * 4 + 4), dtype=torch.uint8, device="cuda")
    return s


# ----------------------------------------------------------- the plain forms

def _rotated(x, pos, freq, layout, mscale):
    """x [T, ..., R] in 32 bits; the angles in 64, since far positions lose theirs in 32."""
    a = pos.double()[:, None] * freq[None]
    half = x.shape[-1] // 2
    shape = [x.shape[0]] + [1] * (x.dim() - 2) + [half]
    c, sn = (a.cos() * mscale).float().view(shape), (a.sin() * mscale).float().view(shape)
    if layout == "half":
        u, v = x[..., :half], x[..., half:]
        return torch.cat([u * c - v * sn, u * sn + v * c], dim=-1)
    u, v = x[..., 0::2], x[..., 1::2]
    return torch.stack([u * c - v * sn, u * sn + v * c], dim=-1).flatten(-2)


def _plain_rope(s):
    s["out"].copy_(_rotated(s["x"].float(), s["pos"], s["freq"], s["case"]["layout"], s["mscale"]))
    return {"out": s["out"]}


def _appended(s):
    c = s["case"]
    if c["kind"] == "bf16":
        got = {"rows": s["cache"].view(torch.bfloat16)}
    elif c["kind"] == "fp8":
        got = {"codes": s["cache"][:, :512].view(torch.float8_e4m3fn), "scales": s["cache"][:, 512:528].view(torch.float32),
               "rope": s["cache"][:, 528:].view(torch.bfloat16)}
    else:
        got = {"codes": s["cache"].view(torch.float8_e4m3fn), "scales": s["scales"]}
    return {**got, "dense": s["rows"]} if c["dense"] else got


def _plain_append(s):
    c, page = s["case"], s["case"]["page"]
    t = torch.arange(s["total"], device="cuda")
    b = torch.searchsorted(s["cu"][1:].long(), t, right=True)
    place = s["lens"].long()[b] - s["cu"].long()[b + 1] + t
    at = s["table"].long()[b, place // page]
    slot = at * page + place % page
    x = s["latent"].float()
    if c["norm"]:
        x = x * (x.square().mean(1, keepdim=True) + EPS).rsqrt() * s["w"].float()
    pos = place if s["pos"] is None else s["pos"]
    row = torch.cat([x, _rotated(s["k_pe"].float(), pos, s["freq"], c["layout"], s["mscale"])], dim=1)
    if c["dense"]:
        s["rows"].copy_(row)
    if c["kind"] == "bf16":
        s["cache"][slot] = row.to(torch.bfloat16).view(torch.uint8)
        return _appended(s)
    if c["kind"] == "fp8":
        v = row[:, :512].reshape(-1, 4, 128)
        top = v.abs().amax(2)
        sc = torch.where(top > 0, top / 448.0, 1.0)
        codes = (v / sc[:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).view(-1, 512)
        s["cache"][slot] = torch.cat([codes, sc.view(torch.uint8), row[:, 512:].to(torch.bfloat16).view(torch.uint8)], dim=1)
        return _appended(s)
    pages, old = s["scales"].numel(), s["scales"]
    top = torch.zeros_like(old).scatter_reduce_(0, at, row.abs().amax(1), "amax")
    first = torch.full((pages,), page, dtype=torch.int64, device="cuda").scatter_reduce_(0, at, place % page, "amin")
    need = _pow2(top)
    new = torch.where(first < page, torch.where(first == 0, need, torch.maximum(old, need)), old)
    codes = s["cache"].view(pages, page, 576)
    grown = torch.nonzero((new > old) & (first > 0) & (first < page)).squeeze(1)  # earlier rows of a page whose scale grows
    was = codes[grown].view(torch.float8_e4m3fn).float()
    earlier = torch.arange(page, device="cuda")[None, :, None] < first[grown][:, None, None]
    codes[grown] = torch.where(earlier, was * (old / new)[grown][:, None, None], was).to(torch.float8_e4m3fn).view(torch.uint8)
    s["cache"][slot] = (row / new[at][:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    old.copy_(new)
    return _appended(s)


def _plain_decode(s):
    c, page = s["case"], s["case"]["page"]
    B, rows = c["B"], c["Hq"] * c["q_len"]
    j = torch.arange(s["most"], device="cuda")
    at = s["table"].long()[:, j // page].clamp(min=0)
    key = s["cache"][at * page + j % page].view(torch.float8_e4m3fn).float().mul_(s["scales"][at][..., None])
    q = torch.cat([s["q_lat"], s["q_pe"]], dim=-1).float().view(B, rows, 576) * SCALE
    last = s["lens"][:, None] - c["q_len"] + torch.arange(rows, device="cuda")[None] // c["Hq"]
    sc = torch.matmul(q, key.transpose(1, 2)).masked_fill_(j[None, None] > last[:, :, None], -math.inf)
    top = sc.amax(2, keepdim=True).clamp(min=-1e30)
    p = sc.sub_(top).exp_()
    total = p.sum(2, keepdim=True)
    s["out"].copy_((torch.matmul(p, key[:, :, :512]) / total.clamp(min=1e-30)).view(s["out"].shape))
    s["lse"].copy_((top + total.log()).view(s["lse"].shape))
    return {"out": s["out"], "lse": s["lse"]}


def run(s):
    c = s["case"]
    if own:
        import mla_latent_kv_cache_gb300 as mla
        if c["op"] == "rope":
            mla.mla_rope(s["x"], s["pos"], s["steps"], s["out"], interleaved=c["layout"] == "interleaved", mscale=s["mscale"])
            return {"out": s["out"]}
        if c["op"] == "append":
            kind = {"bf16": mla.MLA_CACHE_BF16_576, "fp8": mla.MLA_CACHE_FP8_DS_MLA_656, "page8": mla.MLA_CACHE_FP8_PAGE_576}[c["kind"]]
            mla.mla_cache_append(s["latent"], s["k_pe"], s["cu"], s["lens"], s["table"], c["page"], s["cache"], kind,
                                 steps=s["steps"], positions=s["pos"], interleaved=c["layout"] == "interleaved", mscale=s["mscale"],
                                 norm_weight=s["w"], eps=EPS, scales=s["scales"] if c["kind"] == "page8" else None, rows=s["rows"])
            return _appended(s)
        mla.mla_decode_fp8_page(s["q_lat"], s["q_pe"], s["cache"], s["scales"], c["page"], s["table"], s["lens"], c["q_len"], SCALE,
                                s["out"], s["lse"], s["workspace"])
        return {"out": s["out"], "lse": s["lse"]}
    return {"rope": _plain_rope, "append": _plain_append, "decode": _plain_decode}[c["op"]](s)


# ------------------------------------------------- the definitions in 64 bits

def _turned(x, pos, freq, layout, mscale):
    """x [..., R] as complex numbers, each turned by its angle."""
    half = x.shape[-1] // 2
    z = torch.complex(x[..., :half], x[..., half:]) if layout == "half" else torch.view_as_complex(x.unflatten(-1, (half, 2)).contiguous())
    angle = torch.outer(pos.double(), freq)
    z = z * torch.polar(torch.full_like(angle, mscale), angle).view(len(pos), *[1] * (x.dim() - 2), half)
    return torch.cat([z.real, z.imag], dim=-1) if layout == "half" else torch.view_as_real(z).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return {"out": _turned(s["x"].double(), s["pos"], s["freq"], case["layout"], s["mscale"])}
    page = case["page"]
    if case["op"] == "append":
        n, before = _tokens(case)
        kind = case["kind"]
        pool = s["cache"]
        if kind == "fp8":
            got = {"codes": pool[:, :512].view(torch.float8_e4m3fn).double(), "scales": pool[:, 512:528].view(torch.float32).double(),
                   "rope": pool[:, 528:].view(torch.bfloat16).double()}
        else:
            got = {"rows": pool.view(torch.bfloat16).double()} if kind == "bf16" else {
                "codes": pool.view(torch.float8_e4m3fn).double(), "scales": s["scales"].double()}
        if case["dense"]:
            got["dense"] = torch.zeros((s["total"], 576), dtype=torch.float64, device="cuda")
        a = 0
        for b, (m, p) in enumerate(zip(n.tolist(), before.tolist())):
            if m == 0:
                continue
            x = s["latent"][a:a + m].double()
            if case["norm"]:
                x = x / torch.sqrt((x ** 2).sum(1, keepdim=True) / 512 + EPS) * s["w"].double()
            place = torch.arange(p, p + m, device="cuda")
            r = _turned(s["k_pe"][a:a + m].double(), place if s["pos"] is None else s["pos"][a:a + m], s["freq"], case["layout"], s["mscale"])
            row = torch.cat([x, r], dim=1)
            ids = s["table"][b].long()[place // page]
            slot = ids * page + place % page
            if case["dense"]:
                got["dense"][a:a + m] = row
            if kind == "bf16":
                got["rows"][slot] = row
            elif kind == "fp8":
                top = x.unflatten(1, (4, 128)).abs().amax(2) / 448
                got["scales"][slot], got["rope"][slot] = top, r
                got["codes"][slot] = x / top.repeat_interleave(128, dim=1)
            else:
                here, first = s["table"][b].long()[p // page:(p + m - 1) // page + 1], p // page
                top = torch.zeros(len(here), dtype=torch.float64, device="cuda")
                top.index_reduce_(0, place // page - first, row.abs().amax(1), "amax")
                scale = torch.exp2(torch.ceil(torch.log2(top / 448)).clamp(-40, 40))
                if p % page:
                    was = got["scales"][here[0]].item()
                    if was < scale[0].item():
                        got["codes"][here[0] * page:here[0] * page + p % page] *= was / scale[0].item()
                    scale[0] = max(was, scale[0].item())
                got["scales"][here] = scale
                got["codes"][slot] = row / scale[place // page - first][:, None]
            a += m
        return got
    t, Hq, q_len = _tokens(case), case["Hq"], case["q_len"]
    out = torch.zeros((case["B"] * q_len, Hq, 512), dtype=torch.float64, device="cuda")
    lse = torch.full((case["B"] * q_len, Hq), -math.inf, dtype=torch.float64, device="cuda")
    for b, m in enumerate(t.tolist()):
        j = torch.arange(m, device="cuda")
        ids = s["table"][b].long()[j // page]
        key = s["cache"][ids * page + j % page].view(torch.float8_e4m3fn).double() * s["scales"][ids].double()[:, None]
        for i in range(q_len):
            see = m - q_len + i + 1
            if see <= 0:
                continue
            r = b * q_len + i
            z = torch.cat([s["q_lat"][r], s["q_pe"][r]], dim=1).double() @ key[:see].T * SCALE
            lse[r] = torch.logsumexp(z, 1)
            out[r] = torch.softmax(z, 1) @ key[:see, :512]
    return {"out": out, "lse": lse}
