"""Timed cases of the KV-cache and attention operators.

Four operators of a decoder layer's attention, with keys and values held in Q4_0 blocks
in a paged cache:

  qk_kv_append    rotates q and k by position, quantizes k and v, writes them to their pages
  qk_kv_read      reads a range of cached positions back as float values
  qk_attn_paged   attention of new rows over the cache (decode, verification, short chunks)
  qk_attn_prompt  attention over whole packed prompts held as float q, k, v

Each case runs one of them (an append also reads the appended rows back, so that its
output is the values the cache holds).  `run` computes the plain form in elementary torch
operations, or makes the library's calls where `own` is set.

The cache: uint8 [pages][kv heads][page bytes].  One page of one head is K codes
[tokens][D / 2 bytes], K scales f16 [tokens][D / 32], then V the same way.  A code row is
4 groups g of D / 32 dwords b; dword (g, b) holds dims 32 b + 8 g + j, j = 0..7, nibble n
(counted from the low end) being j = 2 n for n < 4 and j = 2 (n - 4) + 1 for n >= 4.
Scale b covers dims 32 b .. 32 b + 31; the value is scale * (code - 8).
"""
import math

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_ES = {"f32": 4, "f16": 2, "bf16": 2}
#: dim offset j of nibble n of a code dword
_NIBBLE_DIM = [0, 2, 4, 6, 1, 3, 5, 7]


# ---------------------------------------------------------------------------
# cases

def _cache_case(name, kind, dtype, n_seq, new_lo, new_hi, past_lo, past_hi, heads, kv_heads, dim, page, **more):
    return {**({"name": name} if name else {}), "kind": kind, "dtype": dtype, "n_seq": n_seq, "new_lo": new_lo, "new_hi": new_hi,
            "past_lo": past_lo, "past_hi": past_hi, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "page": page, **more}


def _prompt_case(name, dtype, n_seq, len_lo, len_hi, heads, kv_heads, dim, causal=True, window=0):
    return {**({"name": name} if name else {}), "kind": "prompt", "dtype": dtype, "n_seq": n_seq, "len_lo": len_lo, "len_hi": len_hi,
            "heads": heads, "kv_heads": kv_heads, "dim": dim, "causal": causal, "window": window}


def listed():
    """Attention widths are those of the 4096-wide layers whose projections the library
    serves (32 heads of 128), with all heads or 8 of them as key / value heads."""
    return [
        # one token of one conversation: launch latency
        _cache_case("append_one", "append", "f32", 1, 1, 1, 300, 300, 32, 8, 128, 16, rot=128, style="halves"),
        # one decode step of a full serving batch, half of each head rotated
        _cache_case("append_batch", "append", "bf16", 64, 1, 1, 100, 4000, 32, 8, 128, 64, rot=64, style="halves"),
        # chunks of several prompts entering the cache, neighbouring dims as pairs
        _cache_case("append_chunk", "append", "f16", 5, 411, 2048, 0, 900, 32, 32, 128, 32, rot=128, style="pairs"),
        # cached prefixes expanded for the next chunk's prompt attention
        _cache_case("read_prefix", "read", "bf16", 3, 2501, 16384, 0, 0, 32, 8, 128, 64),
        # one conversation, short: latency
        _cache_case("paged_one", "paged", "f32", 1, 1, 1, 316, 316, 32, 32, 128, 16, window=0),
        # one conversation, long: the split over the cache fills the card
        _cache_case("paged_long", "paged", "f16", 1, 1, 1, 65501, 65501, 32, 8, 128, 64, window=0),
        # a serving batch of uneven lengths
        _cache_case("paged_batch", "paged", "bf16", 64, 1, 1, 61, 8190, 32, 8, 128, 64, window=0),
        # drafted tokens checked together, small heads, a sliding window
        _cache_case("paged_verify", "paged", "f32", 16, 2, 6, 700, 4099, 32, 8, 64, 32, window=2048),
        # a short question: latency
        _prompt_case("prompt_short", "bf16", 1, 131, 131, 32, 8, 128),
        # several prompts packed, uneven
        _prompt_case("prompt_packed", "bf16", 7, 37, 2047, 32, 8, 128),
        # one long document
        _prompt_case("prompt_long", "f16", 1, 8192, 8192, 32, 8, 128),
        # full-precision activations, all heads their own
        _prompt_case("prompt_f32", "f32", 3, 300, 1500, 32, 32, 64),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["append", "read", "paged", "paged", "prompt", "prompt"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    dim = rng.choice([64, 96, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8, 8, 16, 32])
    heads = kv_heads * rng.choice([g for g in (1, 2, 3, 4, 5, 8, 16) if kv_heads * g <= 32])
    window = rng.choice([0, 0, 0, _log_int(rng, 16, 2048)])
    if kind == "prompt":
        n_seq = _log_int(rng, 1, 24)
        hi = min(_log_int(rng, 1, 2500 if dtype == "f32" else 5000), int(8000 * min(1.0, 128 / dim)) // n_seq)
        return _prompt_case(None, dtype, n_seq, max(1, int(hi * rng.uniform(0.02, 1.0))), hi, heads, kv_heads, dim,
                            causal=rng.random() < 0.8, window=window)
    page = rng.choice([16, 32, 64, 128, 256])
    if kind == "paged":
        n_seq = _log_int(rng, 1, 96)
        new = rng.choice([1, 1, 1, rng.randint(2, 12)])
        past = _log_int(rng, 1, max(2, min(65536, int(2.0e8 / (n_seq * kv_heads * dim)))))
        return _cache_case(None, kind, dtype, n_seq, max(1, new // 2), new, int(past * rng.uniform(0.01, 1.0)), past,
                           heads, kv_heads, dim, page, window=window)
    n_seq = _log_int(rng, 1, 64)
    new = _log_int(rng, 1, max(1, 6000 // n_seq))
    past = _log_int(rng, 1, 4000)
    if kind == "read":
        return _cache_case(None, kind, dtype, n_seq, max(1, new // 3), new, int(past * rng.uniform(0.0, 1.0)), past,
                           heads, kv_heads, dim, page)
    rot = rng.choice([dim, dim, dim // 2])
    return _cache_case(None, kind, dtype, n_seq, max(1, new // 3), new, int(past * rng.uniform(0.0, 1.0)), past, heads,
                       kv_heads, dim, page, rot=rot, style=rng.choice(["halves", "pairs"]))


def _spread(n, lo, hi):
    """n lengths over lo .. hi, the longest first, in no order otherwise."""
    return [hi] + [lo + int((hi - lo + 1) * ((i * 0.6180339887) % 1.0)) for i in range(1, n)]


def _lens(case):
    """(new rows, rows before them) of each sequence."""
    new = _spread(case["n_seq"], case["new_lo"], case["new_hi"])
    past = _spread(case["n_seq"], case["past_lo"], case["past_hi"])
    return new, past


def work(case):
    es, h, hk, dim = _ES[case["dtype"]], case["heads"], case["kv_heads"], case["dim"]
    if case["kind"] == "prompt":
        lens = _spread(case["n_seq"], case["len_lo"], case["len_hi"])
        pairs = sum(_visible(n, 0, case["window"], case["causal"]) for n in lens)
        return {"bytes": sum(lens) * dim * es * (2 * h + 2 * hk), "flops": 4 * dim * h * pairs}
    new, past = _lens(case)
    token = 2 * hk * (dim // 2 + dim // 16)  # a cached position: K and V codes and scales
    if case["kind"] == "paged":
        w = case["window"]
        seen = sum(p + n if w == 0 else min(p + n, n + w - 1) for n, p in zip(new, past))
        pairs = sum(_visible(n, p, w, True) for n, p in zip(new, past))
        return {"bytes": seen * token + 2 * sum(new) * h * dim * es, "flops": 4 * dim * h * pairs}
    rows = sum(new)
    values = 2 * hk * dim
    if case["kind"] == "read":
        return {"bytes": rows * (token + values * es), "flops": rows * values}
    read_in = (values + h * dim) * es + case["rot"] * 4
    return {"bytes": rows * (read_in + h * dim * es + 2 * token + values * es),
            "flops": rows * ((hk + h) * case["rot"] * 3 + 3 * values)}


def _visible(n, past, window, causal):
    """(row, position) pairs that n new rows after `past` positions attend to."""
    total = 0
    for i in range(n):
        at = past + i
        hi = at + 1 if causal else past + n
        lo = 0 if window == 0 else max(0, at - window + 1)
        total += hi - lo
    return total


# ---------------------------------------------------------------------------
# inputs

def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _cu(lens):
    return _int32([0] + list(np.cumsum(lens)))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 7919 + 17)
    dt, h, hk, dim = _DT[case["dtype"]], case["heads"], case["kv_heads"], case["dim"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)

    # a few channels of the keys are larger than the rest, as in trained models
    channel = torch.exp(0.4 * normal(hk, dim))
    s = {"kind": case["kind"], "dim": dim, "scale": 1.0 / math.sqrt(dim)}
    if case["kind"] == "prompt":
        lens = _spread(case["n_seq"], case["len_lo"], case["len_hi"])
        n = sum(lens)
        s |= {"q": normal(n, h, dim).to(dt), "k": (normal(n, hk, dim) * channel).to(dt), "v": normal(n, hk, dim).to(dt),
              "cu": _cu(lens), "causal": case["causal"], "window": case["window"]}
        return s
    new, past = _lens(case)
    page, n = case["page"], sum(new)
    need = [-(-(a + b) // page) for a, b in zip(new, past)]
    n_pages = sum(need) + 5
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32).cpu().numpy()
    table = np.zeros((len(new), max(need) + 1), np.int32)
    at = 0
    for i, m in enumerate(need):
        table[i, :m] = order[at:at + m]
        at += m
    half = page * (dim // 2 + dim // 16)
    pages = torch.randint(0, 256, (n_pages, hk, 2 * half), generator=gen, device="cuda", dtype=torch.uint8)
    for base in (0, half):
        sc = pages[:, :, base + page * dim // 2:base + half].view(torch.float16)
        d = (0.12 + 0.25 * torch.rand(sc.shape, generator=gen, device="cuda"))
        d *= torch.where(torch.rand(sc.shape, generator=gen, device="cuda") < 0.5, -1.0, 1.0)
        sc.copy_(d.to(torch.float16))
    s |= {"pages": pages, "page": page, "table": torch.from_numpy(table).cuda(), "cu": _cu(new), "start": _int32(past),
          "n": n, "dt": dt}
    if case["kind"] == "paged":
        s |= {"q": normal(n, h, dim).to(dt), "window": case["window"], "most": max(new)}
    if case["kind"] == "append":
        rot = case["rot"]
        angle = torch.arange(max(a + b for a, b in zip(new, past)) + 1, dtype=torch.float64, device="cuda")[:, None]
        angle = angle * 10000.0 ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64, device="cuda") / rot)
        s |= {"q": normal(n, h, dim).to(dt), "k": (normal(n, hk, dim) * channel).to(dt), "v": normal(n, hk, dim).to(dt),
              "rope": torch.stack([angle.cos(), angle.sin()], -1).to(torch.float32), "style": case["style"]}
    return s


# ---------------------------------------------------------------------------
# the calls, and the plain forms

def run(s):
    kind = s["kind"]
    if own:
        import quantized_gemv_quantize_amd as qk
        if kind == "prompt":
            return qk.qk_attn_prompt(s["q"], s["k"], s["v"], s["cu"], scale=s["scale"], causal=s["causal"],
                                     window=s["window"])
        cache = (s["pages"], s["page"], s["table"], s["cu"], s["start"])
        if kind == "paged":
            return qk.qk_attn_paged(*cache, s["q"], scale=s["scale"], window=s["window"])
        if kind == "read":
            return qk.qk_kv_read(*cache, s["n"], s["dim"], dtype=s["dt"])
        style = qk.QK_ROPE_HALVES if s["style"] == "halves" else qk.QK_ROPE_PAIRS
        q = qk.qk_kv_append(*cache, s["k"], s["v"], q=s["q"], rope=s["rope"], rope_style=style)
        return (q, *qk.qk_kv_read(*cache, s["n"], s["dim"], dtype=s["dt"]))
    if kind == "prompt":
        return _plain_prompt(s)
    if kind == "paged":
        return _plain_paged(s)
    if kind == "read":
        return _plain_read(s)
    q = _plain_append(s)
    return (q, *_plain_read(s))


def _rows(s):
    """(sequence, position) of every new row."""
    row = torch.arange(s["n"], device="cuda")
    seq = torch.searchsorted(s["cu"].long(), row, right=True) - 1
    return seq, s["start"].long()[seq] + row - s["cu"].long()[seq]


def _planes(s):
    """Views of the cache: [codes, scales] of K and of V, codes uint8 [pages][heads][tokens][4 g][D / 32 b][4 bytes]."""
    page, dim, out = s["page"], s["dim"], []
    half = page * (dim // 2 + dim // 16)
    for base in (0, half):
        codes = s["pages"][:, :, base:base + page * dim // 2].unflatten(2, (page, 4, dim // 32, 4))
        scales = s["pages"][:, :, base + page * dim // 2:base + half].view(torch.float16).unflatten(2, (page, dim // 32))
        out.append((codes, scales))
    return out


def _values(codes, scales):
    """f32 [..., D] of code rows [..., 4, D / 32, 4] and scales [..., D / 32]."""
    shift = torch.tensor([0, 4], dtype=torch.uint8, device="cuda")
    nib = ((codes[..., None] >> shift) & 15).flatten(-2)  # [..., g, b, nibble]
    order = torch.tensor([_NIBBLE_DIM.index(j) for j in range(8)], device="cuda")
    code = nib[..., order].transpose(-3, -2).flatten(-2)  # [..., b, 32]
    return ((code.float() - 8.0) * scales.float()[..., None]).flatten(-2)


def _rotate(x, cs, style):
    """x f32 [n][heads][D], cs f32 [n][rot / 2][2]; every operation rounded on its own."""
    rot = 2 * cs.shape[1]
    c, t = cs[:, None, :, 0], cs[:, None, :, 1]
    if style == "halves":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    ac, bs, at, bc = a * c, b * t, a * t, b * c
    if style == "halves":
        turned = torch.cat([ac - bs, at + bc], -1)
    else:
        turned = torch.stack([ac - bs, at + bc], -1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_append(s):
    seq, pos = _rows(s)
    page = s["table"].long()[seq, pos // s["page"]]
    slot = pos % s["page"]
    cs = s["rope"][pos]
    order = torch.tensor(_NIBBLE_DIM, device="cuda")
    for x, (codes, scales) in zip((_rotate(s["k"].float(), cs, s["style"]), s["v"].float()), _planes(s)):
        x = x.unflatten(-1, (-1, 32))
        size = x.abs()
        top = size.amax(-1, keepdim=True)
        lane = torch.arange(32, device="cuda").expand_as(x)
        first = torch.where(size == top, lane, 32).amin(-1, keepdim=True)  # ties: the first of them
        d = torch.gather(x, -1, first) / -8.0
        inv = torch.where(d != 0, 1.0 / d, torch.zeros_like(d))
        code = (x * inv + 8.5).trunc().clamp(max=15).to(torch.uint8)  # [n, heads, b, 32]
        nib = code.unflatten(-1, (4, 8)).transpose(-3, -2)[..., order]  # [n, heads, g, b, nibble]
        codes[page, :, slot] = nib[..., 0::2] | (nib[..., 1::2] << 4)
        scales[page, :, slot] = d[..., 0].to(torch.float16)
    return _rotate(s["q"].float(), cs, s["style"]).to(s["dt"])


def _plain_read(s):
    seq, pos = _rows(s)
    page = s["table"].long()[seq, pos // s["page"]]
    slot = pos % s["page"]
    return tuple(_values(codes[page, :, slot], scales[page, :, slot]).to(s["dt"]) for codes, scales in _planes(s))


def _softmax_values(score, seen, v):
    score = torch.where(seen, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / torch.where(total == 0, torch.ones_like(total), total)


def _plain_paged(s):
    """All rows of all sequences padded to the longest: [sequence, kv head, new row x group, position]."""
    (kc, ks), (vc, vs) = _planes(s)
    table = s["table"].long()
    k, v = (_values(c[table], d[table]).transpose(2, 3) for c, d in ((kc, ks), (vc, vs)))  # [B, pages, tokens, heads, D]
    b, hk, dim = table.shape[0], k.shape[3], s["dim"]
    k, v = (x.flatten(1, 2).transpose(1, 2) for x in (k, v))  # [B, heads, positions, D]
    n, h = s["q"].shape[:2]
    new = (s["cu"][1:] - s["cu"][:-1]).long()
    seq, pos = _rows(s)
    at = pos - s["start"].long()[seq]
    most = s["most"]
    q = torch.zeros(b, most, h, dim, device="cuda")
    q[seq, at] = s["q"].float()
    q = q.unflatten(2, (hk, h // hk)).transpose(1, 2).flatten(2, 3)  # [B, heads, row x group, D]
    score = torch.matmul(q, k.transpose(-1, -2).contiguous()) * s["scale"]
    here = (s["start"].long()[:, None] + torch.arange(most, device="cuda")).repeat_interleave(h // hk, 1)[:, None, :, None]
    where = torch.arange(k.shape[2], device="cuda")
    seen = (where <= here) & (where < (s["start"].long() + new)[:, None, None, None])
    if s["window"]:
        seen = seen & (where > here - s["window"])
    out = _softmax_values(score, seen, v.contiguous())
    out = out.unflatten(2, (most, h // hk)).transpose(1, 2).flatten(2, 3)
    return out[seq, at].to(s["q"].dtype)


def _plain_prompt(s):
    """All packed rows against all packed rows; a pair counts where both are of one sequence."""
    q, k, v = (x.float().transpose(0, 1) for x in (s["q"], s["k"], s["v"]))
    n, g = q.shape[1], q.shape[0] // k.shape[0]
    row = torch.arange(n, device="cuda")
    seq = torch.searchsorted(s["cu"].long(), row, right=True)
    seen = seq[:, None] == seq
    if s["causal"]:
        seen = seen & (row[:, None] >= row)
    if s["window"]:
        seen = seen & (row > row[:, None] - s["window"])
    q = q.unflatten(0, (-1, g))
    score = torch.matmul(q, k.transpose(-1, -2).contiguous()[:, None]) * s["scale"]
    out = _softmax_values(score, seen, v.contiguous()[:, None])
    return out.flatten(0, 1).transpose(0, 1).to(s["q"].dtype)


# ---------------------------------------------------------------------------
# the definitions in 64 bits

def _unpacked(s, at):
    """f64 K and V [positions][heads][D] at page / slot pairs `at`, byte by byte from the layout."""
    page, dim = s["page"], s["dim"]
    half = page * (dim // 2 + dim // 16)
    d = torch.arange(dim, device="cuda")
    block, group, j = d // 32, d % 32 // 8, d % 8
    nibble = j // 2 + 4 * (j % 2)
    byte = (group * (dim // 32) + block) * 4 + nibble // 2
    out = []
    for base in (0, half):
        raw = s["pages"][at[0]]  # [positions, heads, bytes]
        code_at = base + at[1][:, None] * (dim // 2) + byte
        code = torch.gather(raw, 2, code_at[:, None].expand(-1, raw.shape[1], -1))
        code = (code >> (4 * (nibble % 2)).to(torch.uint8)) & 15
        sc_at = base + page * dim // 2 + 2 * (at[1][:, None] * (dim // 32) + block)
        lo, hi = (torch.gather(raw, 2, (sc_at + i)[:, None].expand(-1, raw.shape[1], -1)) for i in (0, 1))
        sc = torch.stack([lo, hi], -1).view(torch.float16)[..., 0]
        out.append(sc.double() * (code.double() - 8))
    return out


def _one_row_block(q, k, v, scale, first_at, causal, window):
    """f64 attention of rows at first_at .. against positions 0 .. of one head."""
    at = first_at + torch.arange(q.shape[0], device="cuda")[:, None]
    pos = torch.arange(k.shape[0], device="cuda")[None]
    hide = torch.zeros(q.shape[0], k.shape[0], dtype=torch.bool, device="cuda")
    if causal:
        hide |= pos > at
    if window:
        hide |= pos <= at - window
    score = (q @ k.T) * scale
    score.masked_fill_(hide, -math.inf)
    return torch.softmax(score, -1) @ v


def exact(case, seed):
    s = prepare(case, seed)
    kind, dim, h, hk = case["kind"], case["dim"], case["heads"], case["kv_heads"]
    cu = s["cu"].tolist()
    if kind in ("prompt", "paged"):
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        for b in range(len(cu) - 1):
            rows = slice(cu[b], cu[b + 1])
            if kind == "prompt":
                k, v, first, causal = s["k"][rows].double(), s["v"][rows].double(), 0, s["causal"]
            else:
                first, causal = int(s["start"][b]), True
                pos = torch.arange(first + cu[b + 1] - cu[b], device="cuda")
                k, v = _unpacked(s, (s["table"][b].long()[pos // s["page"]], pos % s["page"]))
            for i in range(h):
                g = i // (h // hk)
                out[rows, i] = _one_row_block(s["q"][rows, i].double(), k[:, g], v[:, g], 1.0 / math.sqrt(dim), first,
                                              causal, s["window"])
        return out
    at = [(b, int(s["start"][b]) + i) for b in range(len(cu) - 1) for i in range(cu[b + 1] - cu[b])]
    seq, pos = (torch.tensor(x, device="cuda") for x in zip(*at))
    if kind == "read":
        return tuple(_unpacked(s, (s["table"].long()[seq, pos // s["page"]], pos % s["page"])))
    half = case["rot"] // 2
    i = torch.arange(half, device="cuda")
    lo, hi = (i, i + half) if case["style"] == "halves" else (2 * i, 2 * i + 1)
    turn = torch.complex(s["rope"][..., 0].double(), s["rope"][..., 1].double())[pos][:, None]

    def rotated(x):
        y = x.double().clone()
        z = torch.complex(y[..., lo], y[..., hi]) * turn
        y[..., lo], y[..., hi] = z.real, z.imag
        return y

    def stored(x):
        y = x.reshape(*x.shape[:-1], dim // 32, 32)
        up, down = y.max(-1).values, y.min(-1).values
        first_up = torch.where(y == up[..., None], 1, 0).argmax(-1)
        first_down = torch.where(y == down[..., None], 1, 0).argmax(-1)
        most = torch.where((up > -down) | ((up == -down) & (first_up < first_down)), up, down)
        d = most / -8
        code = torch.floor(torch.where(d[..., None] == 0, 0.0, y / d[..., None]) + 8.5).clamp(0, 15)
        return (d.to(torch.float16).double()[..., None] * (code - 8)).reshape(x.shape)

    return rotated(s["q"]), stored(rotated(s["k"])), stored(s["v"].double())
