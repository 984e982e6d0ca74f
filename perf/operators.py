"""Measured cases of the 4-bit (E2M1) KV-cache operators.

Three operators over one cache format: the quantising write
(``pkv_write_e2m1``), the read of cached rows (``pkv_read_e2m1``) and attention
of a flat variable-length batch over the cache (``pkv_attention_varlen_e2m1``,
and ``pkv_write_attention_varlen_e2m1``, which writes and attends).

The format: K and V are one uint8 tensor each, [num_blocks, num_kv_heads,
9 * head_dim].  The 9 * head_dim bytes of a (block, head) are its 16 tokens' rows
of head_dim / 2 code bytes (element 2 i in the low nibble of byte i, 2 i + 1 in
the high one), then its 16 tokens' rows of head_dim / 16 scale bytes.  A code is E2M1 (sign,
two exponent bits of bias 1, one mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6), a
scale is E4M3, one for 16 consecutive elements, and each tensor has one fp32
scale t: an element stands for t * scale * code.

The write of a row x takes y = x / t (rounded to fp32); a block's scale is
max|y| / 6 (rounded to fp32) rounded to E4M3, at most 448; its codes are
y / scale (rounded to fp32) rounded to E2M1, at most 6, and 0 under a scale of 0.
All roundings are to nearest, ties to even.
"""

import math
import random

import torch

own = False

BLOCK = 16


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
# op: "attend" (attention alone), "step" (write of the new tokens, then
#   attention), "write" (write of new tokens and the read of what they became),
#   "read" (rows of whole contexts).
# requests have `new` tokens each (the first one `first`, where that is not 0)
# on top of lo..hi cached tokens, drawn with `mix`; heads are hq / hkv of d.
def _case(name, op, requests, new, lo, hi, hq, hkv, d, first=0, window=0, causal=True, lse=False,
          dtype="bf16", mix=0):
    c = {"op": op, "requests": requests, "new": new, "first": first, "lo": lo, "hi": hi,
         "hq": hq, "hkv": hkv, "d": d, "window": window, "causal": causal, "lse": lse,
         "dtype": dtype, "mix": mix}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one user's next token on a long document: few rows, latency
        _case("decode_1x8k", "attend", 1, 1, 8191, 8191, 32, 8, 128),
        # a serving step at batch 64: every request's new token written, then attended
        _case("step_64", "step", 64, 1, 511, 4095, 32, 8, 128, mix=1),
        # the smallest step: three short requests, one with no cached token
        _case("step_tiny", "step", 3, 1, 0, 40, 2, 1, 64, lse=True, mix=2),
        # two very long contexts
        _case("decode_2x128k", "attend", 2, 1, 131001, 131070, 32, 8, 128, mix=3),
        # speculated tokens (three each) of 16 requests with one KV head, under a
        # sliding window, with the log-sum-exps that a later merge wants
        _case("tails_16", "attend", 16, 3, 100, 9000, 16, 1, 128, window=1024, lse=True, mix=4),
        # a chunk of a prompt on its cached beginning, among decoding requests
        _case("mixed_chunk", "step", 32, 1, 256, 1001, 32, 8, 128, first=1024, mix=5),
        # a whole prompt in one chunk
        _case("prefill_8k", "attend", 1, 8192, 0, 0, 32, 8, 128),
        # ragged prompts, three query heads to a KV head, heads of 64
        _case("prefill_ragged", "step", 5, 130, 0, 333, 12, 4, 64, first=777, mix=6),
        # a decode step's 64 tokens, as they were written
        _case("write_64", "write", 64, 1, 5, 2047, 8, 8, 128, mix=7),
        # a prompt's 8192 tokens written and handed on as bf16
        _case("write_8k", "write", 1, 8192, 0, 0, 8, 8, 128),
        # fp32 states of odd prompts, three heads of 64
        _case("write_f32", "write", 7, 61, 3, 90, 3, 3, 64, first=501, dtype="f32", mix=8),
        # 64 whole contexts read back, as for moving requests to another cache
        _case("read_64", "read", 64, 0, 512, 4096, 8, 8, 128, mix=9),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["attend", "attend", "step", "step", "write", "read"])
        hkv = rng.choice([1, 2, 3, 4, 8])
        group = rng.choice([1, 2, 3, 4, 7, 8, 16]) if op in ("attend", "step") else 1
        d = rng.choice([64, 128])
        requests = _log_int(rng, 1, 64)
        hi = _log_int(rng, 16, 131072)
        lo = rng.randint(0, hi)
        first, new, dtype = 0, 0, "bf16"
        if op in ("attend", "step"):
            new = rng.choice([1, 1, 1, 2, 3, 4, rng.randint(5, 40)])
            if rng.random() < 0.4:
                first = _log_int(rng, 5, 8192)
        elif op == "write":
            new = _log_int(rng, 1, 512)
            first = _log_int(rng, 1, 8192)
            dtype = rng.choice(["bf16", "f32"])
        else:
            dtype = rng.choice(["bf16", "f32"])
            lo, hi = max(lo, 1), max(hi, 1)
        window = rng.choice([0, 0, 0, _log_int(rng, 16, 4096)]) if op == "attend" else 0
        causal = not (op == "attend" and window == 0 and rng.random() < 0.2)
        c = _case("", op, requests, new, lo, hi, group * hkv, hkv, d, first=first, window=window,
                  causal=causal, lse=rng.random() < 0.3, dtype=dtype, mix=rng.randint(10, 1 << 20))
        lens = _lens(c)
        most_l, most_n = max(computed + n for computed, n in lens), max(n for _, n in lens)
        if op in ("attend", "step") and requests * most_n * most_l * c["hq"] > 32 * 8192 * 8192 // 2:
            continue            # the plain form's scores: no more than the largest listed case
        if requests * most_l * hkv * d > 64 * 4096 * 8 * 128:
            continue            # cached elements, padded: no more than the largest listed case
        return c


def _lens(case):
    """(cached tokens, new tokens) of each request."""
    rng = random.Random(case["mix"])
    out = []
    for r in range(case["requests"]):
        n = case["first"] if r == 0 and case["first"] else case["new"]
        out.append((rng.randint(case["lo"], case["hi"]), n))
    return out


# ---------------------------------------------------------------------------
# the format, in torch
# ---------------------------------------------------------------------------
def _quantise(x, t):
    """fp32 rows [..., d] -> code bytes [..., d / 2] and scale bytes [..., d / 16]."""
    full = lambda v: torch.full((), v, dtype=torch.float32, device=x.device)  # noqa: E731
    y = (x / full(t)).unflatten(-1, (-1, 16))
    scale = (y.abs().amax(-1) / full(6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = scale.to(torch.float32).unsqueeze(-1)
    m = torch.where(s > 0, y / s, torch.zeros_like(y))
    a = m.abs()
    code = (a > 0.25).to(torch.uint8)
    code += a >= 0.75
    code += a > 1.25
    code += a >= 1.75
    code += a > 2.5
    code += a >= 3.5
    code += a > 5.0
    code += (m < 0) * 8
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale.view(torch.uint8)


def _values(codes, scales, t):
    """Code and scale bytes -> fp32 rows."""
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    e, m = ((n >> 1) & 3).float(), (n & 1).float()
    v = torch.where(e > 0, (1 + 0.5 * m) * torch.exp2(e - 1), 0.5 * m)
    v = torch.where(n > 7, -v, v)
    s = scales.view(torch.float8_e4m3fn).to(torch.float32).unsqueeze(-1)
    return (v.unflatten(-1, (-1, 16)) * s).flatten(-2) * t


def _parts(cache, d):
    """Views of a cache: codes [blocks, heads, 16, d / 2], scales [blocks, heads, 16, d / 16]."""
    return (cache[..., :8 * d].unflatten(-1, (16, d // 2)),
            cache[..., 8 * d:].unflatten(-1, (16, d // 16)))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    lens = _lens(case)
    counts = [-(-(c + n) // BLOCK) for c, n in lens]
    need = sum(counts)
    num_blocks = need + need // 8 + 1
    perm = torch.randperm(num_blocks, generator=g, device=dev)
    # channels of unlike size, as keys and values have
    gain = torch.exp(0.5 * torch.randn(2, hkv, 1, d, generator=g, device=dev))
    t = (0.5, 0.75)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    def filled(which):
        cache = torch.empty(num_blocks, hkv, 9 * d, dtype=torch.uint8, device=dev)
        codes, scales = _parts(cache, d)
        for b in range(0, num_blocks, 4096):
            n = min(4096, num_blocks - b)
            x = (normal(n, hkv, 16, d) * gain[which]).bfloat16().float()
            codes[b:b + n], scales[b:b + n] = _quantise(x, t[which])
        return cache

    s = {"op": case["op"], "d": d, "k_scale": t[0], "v_scale": t[1],
         "k_cache": filled(0), "v_cache": filled(1)}
    # the step's metadata, as a runner builds it on the host and copies it over
    table = torch.zeros(len(lens), max(counts + [1]), dtype=torch.int64, device=dev)
    at = 0
    for r, k in enumerate(counts):
        table[r, :k] = perm[at:at + k]
        at += k
    read = case["op"] == "read"
    tokens = [(r, c + i) for r, (c, n) in enumerate(lens) for i in range(n)]
    if read:
        tokens = [(r, p) for r, (c, _) in enumerate(lens) for p in range(c)]
    tok = torch.tensor(tokens, dtype=torch.int64).reshape(-1, 2).to(dev)
    s["slots"] = (table[tok[:, 0], tok[:, 1] // BLOCK] * BLOCK + tok[:, 1] % BLOCK).contiguous()
    kind = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    if case["op"] in ("step", "write"):
        s["k_new"] = (normal(len(tokens), hkv, d) * gain[0, :, 0]).to(kind)
        s["v_new"] = (normal(len(tokens), hkv, d) * gain[1, :, 0]).to(kind)
    if case["op"] in ("write", "read"):
        s["k_out"] = torch.empty(len(tokens), hkv, d, dtype=kind, device=dev)
        s["v_out"] = torch.empty(len(tokens), hkv, d, dtype=kind, device=dev)
        return s
    s["q"] = normal(len(tokens), hq, d).bfloat16()
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(len(tokens), hq, device=dev) if case["lse"] else None
    starts = [0]
    for _, n in lens:
        starts.append(starts[-1] + n)
    s["query_start_loc"] = torch.tensor(starts, dtype=torch.int32).to(dev)
    s["seq_lens"] = torch.tensor([c + n for c, n in lens], dtype=torch.int32).to(dev)
    s["block_table"] = table.to(torch.int32)
    s["max_query_len"] = max(n for _, n in lens)
    s["max_seq_len"] = max(c + n for c, n in lens)
    s["softmax_scale"] = 1.0 / math.sqrt(d)
    s["causal"], s["window"] = case["causal"], case["window"]
    s["flag"] = torch.zeros(1, dtype=torch.int32, device=dev)
    # the scratch that a serving program keeps for its steps
    s["workspace"] = torch.empty(64 << 20, dtype=torch.uint8, device=dev)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    return _kernels(s) if own else _plain(s)


def _kernels(s):
    import paged_kv_attention_17_gb300 as pkv
    scales = (s["k_scale"], s["v_scale"])
    cache = (s["k_cache"], s["v_cache"])
    if s["op"] == "write":
        pkv.pkv_write_e2m1(s["k_new"], s["v_new"], s["slots"], *cache, *scales)
    if s["op"] in ("write", "read"):
        pkv.pkv_read_e2m1(*cache, s["slots"], s["k_out"], s["v_out"], *scales)
        return s["k_out"], s["v_out"]
    batch = (s["query_start_loc"], s["seq_lens"], s["block_table"], s["max_query_len"],
             s["max_seq_len"], s["softmax_scale"])
    more = dict(causal=s["causal"], window=s["window"], workspace=s["workspace"],
                lse_out=s["lse"], error_flag=s["flag"])
    if s["op"] == "step":
        pkv.pkv_write_attention_varlen_e2m1(s["k_new"], s["v_new"], s["slots"], s["q"], *cache,
                                            s["out"], *batch, *scales, **more)
    else:
        pkv.pkv_attention_varlen_e2m1(s["q"], *cache, s["out"], *batch, *scales, **more)
    return (s["out"], s["lse"]) if s["lse"] is not None else s["out"]


def _plain(s):
    d = s["d"]
    if s["op"] in ("step", "write"):
        blk, off = s["slots"] // BLOCK, s["slots"] % BLOCK
        for new, cache, t in ((s["k_new"], s["k_cache"], s["k_scale"]),
                              (s["v_new"], s["v_cache"], s["v_scale"])):
            codes, scales = _parts(cache, d)
            codes[blk, :, off], scales[blk, :, off] = _quantise(new.float(), t)
    if s["op"] in ("write", "read"):
        blk, off = s["slots"] // BLOCK, s["slots"] % BLOCK
        for out, cache, t in ((s["k_out"], s["k_cache"], s["k_scale"]),
                              (s["v_out"], s["v_cache"], s["v_scale"])):
            codes, scales = _parts(cache, d)
            out.copy_(_values(codes[blk, :, off], scales[blk, :, off], t))
        return s["k_out"], s["v_out"]
    return _plain_attention(s)


def _plain_attention(s):
    """Every request padded to the longest: rows [R, n, hq, d], keys [R, hkv, L, d]."""
    q, d, dev = s["q"], s["d"], s["q"].device
    table, lens = s["block_table"].long(), s["seq_lens"].long()
    starts = s["query_start_loc"].long()
    R, n, L = len(lens), s["max_query_len"], s["max_seq_len"]
    hkv = s["k_cache"].shape[1]
    group = q.shape[1] // hkv
    counts = starts[1:] - starts[:-1]

    def keys(cache, t):
        codes, scales = _parts(cache[table[:, :-(-L // BLOCK)]], d)      # [R, blocks, hkv, 16, .]
        x = _values(codes, scales, t)
        return x.transpose(1, 2).flatten(2, 3)[:, :, :L]                 # [R, hkv, L, d]

    i = torch.arange(n, device=dev)
    row = torch.minimum(starts[:-1, None] + i, starts[1:, None] - 1).clamp(min=0)    # [R, n]
    rows = q[row].float().unflatten(2, (hkv, group)).permute(0, 2, 3, 1, 4)          # [R, hkv, group, n, d]
    score = rows.flatten(2, 3) @ keys(s["k_cache"], s["k_scale"]).transpose(2, 3)    # [R, hkv, group n, L]
    score *= s["softmax_scale"]
    j = torch.arange(L, device=dev)
    at = (lens - counts)[:, None] + i                                    # position of each row
    hidden = j >= lens[:, None, None]
    if s["causal"]:
        hidden = hidden | (j > at[:, :, None])
    if s["window"]:
        hidden = hidden | (j <= at[:, :, None] - s["window"])
    hidden = hidden.expand(R, n, L)
    score.view(R, hkv, group, n, L).masked_fill_(hidden[:, None, None], float("-inf"))
    top = score.amax(-1, keepdim=True)
    p = score.sub_(top.clamp(min=-3e38)).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p @ keys(s["v_cache"], s["v_scale"])) / total.clamp(min=1e-38)
    o = o.unflatten(2, (group, n)).permute(0, 3, 1, 2, 4).flatten(2, 3)  # [R, n, hq, d]
    real = i < counts[:, None]
    s["out"].copy_(o[real].to(s["out"].dtype))
    if s["lse"] is None:
        return s["out"]
    lse = (top + total.log()).squeeze(-1).unflatten(2, (group, n)).permute(0, 3, 1, 2).flatten(2, 3)
    s["lse"].copy_(lse[real])
    return s["out"], s["lse"]


# ---------------------------------------------------------------------------
# the work of one pass
# ---------------------------------------------------------------------------
def work(case):
    hq, hkv, d, lens = case["hq"], case["hkv"], case["d"], _lens(case)
    page_row = 2 * hkv * d * 9 / 16                   # K and V of one cached token
    wide = 2 * hkv * d * (4 if case["dtype"] == "f32" else 2)
    new = sum(n for _, n in lens)
    if case["op"] == "write":
        return {"bytes": new * (2 * wide + 2 * page_row + 16), "flops": 0}
    if case["op"] == "read":
        rows = sum(c for c, _ in lens)
        return {"bytes": rows * (wide + page_row + 8), "flops": 0}
    seen, pairs = 0, 0
    for c, n in lens:
        total, w = c + n, case["window"]
        first = 0                                     # the first key that any row sees
        if w:
            first = max(0, c - w + 1)
        seen += total - first
        if not case["causal"]:
            pairs += n * total
        elif not w:
            pairs += n * c + n * (n + 1) // 2
        else:
            pairs += sum(min(c + i + 1, w) for i in range(n))
    size = seen * page_row + 2 * new * hq * d * 2 + seen / BLOCK * 4
    if case["op"] == "step":
        size += new * (2 * hkv * d * 2 + 8)           # (what it writes is what it then reads)
    if case["lse"]:
        size += new * hq * 4
    return {"bytes": size, "flops": 4 * d * hq * pairs}


# ---------------------------------------------------------------------------
# the definition, in 64 bits
# ---------------------------------------------------------------------------
_MAGNITUDES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _exact_row(x, t):
    """What the rows x become in the cache: the format's fp32 and E4M3 roundings
    of quotients that are taken in 64 bits."""
    y = (x.double() / t).float().double().unflatten(-1, (-1, 16))
    a = (y.abs().amax(-1) / 6).float().double()
    _, e = torch.frexp(a)
    step = torch.exp2((e.double() - 4).clamp(min=-9.0))            # 3 mantissa bits, 2^-9 at least
    s = (torch.round(a / step) * step).clamp(max=448.0).unsqueeze(-1)
    z = torch.where(s > 0, (y / s.clamp(min=2.0 ** -9)).float().double(), 0.0 * y)
    mags = torch.tensor(_MAGNITUDES, dtype=torch.float64, device=x.device)
    mids = (mags[1:] + mags[:-1]) / 2
    up, down = torch.searchsorted(mids, z.abs(), right=True), torch.searchsorted(mids, z.abs())
    code = torch.where(up % 2 == 0, up, down)                      # a tie: the even one of the two
    return (torch.sign(z) * mags[code] * s).flatten(-2) * t


def _exact_cache(cache, slots, d, t):
    """Rows of the cache in 64 bits: [rows, heads, d]."""
    page = cache[slots // BLOCK]
    off = (slots % BLOCK).view(-1, 1, 1)
    at = torch.arange(d // 2, device=cache.device)
    codes = page.gather(2, (off * (d // 2) + at).expand(-1, page.shape[1], -1)).long()
    at = torch.arange(d // 16, device=cache.device)
    scales = page.gather(2, (8 * d + off * (d // 16) + at).expand(-1, page.shape[1], -1)).long()
    table = torch.tensor(_MAGNITUDES + [-m for m in _MAGNITUDES], dtype=torch.float64, device=cache.device)
    x = torch.stack([table[codes % 16], table[codes // 16]], -1).flatten(-2)
    e, m = (scales // 8).double(), (scales % 8).double()
    s = torch.where(e > 0, (1 + m / 8) * torch.exp2(e - 7), m * 2.0 ** -9)
    return (x.unflatten(-1, (-1, 16)) * s.unsqueeze(-1)).flatten(-2) * t


def exact(case, seed):
    s = prepare(case, seed)
    d = case["d"]
    if case["op"] == "write":
        return _exact_row(s["k_new"], s["k_scale"]), _exact_row(s["v_new"], s["v_scale"])
    if case["op"] == "read":
        return (_exact_cache(s["k_cache"], s["slots"], d, s["k_scale"]),
                _exact_cache(s["v_cache"], s["slots"], d, s["v_scale"]))
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    group, start = case["hq"] // case["hkv"], 0
    for r, (c, n) in enumerate(_lens(case)):
        p = torch.arange(c + n, device="cuda")
        slots = s["block_table"][r].long()[p // BLOCK] * BLOCK + p % BLOCK
        k = _exact_cache(s["k_cache"], slots, d, s["k_scale"])
        v = _exact_cache(s["v_cache"], slots, d, s["v_scale"])
        if case["op"] == "step":
            k[c:] = _exact_row(s["k_new"][start:start + n], s["k_scale"])
            v[c:] = _exact_row(s["v_new"][start:start + n], s["v_scale"])
        for h in range(case["hq"]):
            for i in range(0, n, 1024):
                row = torch.arange(i, min(i + 1024, n), device="cuda")
                most = c + int(row[-1]) + 1 if case["causal"] else c + n
                x = s["q"][start + row, h].double() @ k[:most, h // group].T * s["softmax_scale"]
                at = (c + row)[:, None]
                if case["causal"]:
                    x[p[:most] > at] = float("-inf")
                if case["window"]:
                    x[p[:most] <= at - case["window"]] = float("-inf")
                w = torch.softmax(x, -1)
                out[start + row, h] = w @ v[:most, h // group]
                lse[start + row, h] = torch.logsumexp(x, -1)
        start += n
    return (out, lse) if case["lse"] else out
