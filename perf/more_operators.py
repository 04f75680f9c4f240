"""Workloads of the dense serving operators over the 4-bit paged KV cache: appending a step's tokens (norm and
rotation of queries and keys, keys and values quantised into their pages, in one call), and attention of each
sequence's new tokens over what it has cached, everything that is visible or a sliding window with the first
tokens (sinks).

Every case has a plain form (elementary torch operations, float32) and, with ``own`` set, the calls that a
user makes of the library.  ``listed()`` gives the named cases, ``draw(rng)`` one more of the same ranges,
``prepare`` the inputs, ``run`` one pass, ``exact`` the same outputs in 64 bits.

Cache format: the entry of a position holds, for each KV head, D/2 bytes of K codes, D/2 of V codes, D/16 of
K scales and D/16 of V scales, padded to 16 bytes; element 2i of a vector is the low nibble of byte i; scales
are float8_e4m3fn, one per 16 elements; codes are E2M1 (0 .5 1 1.5 2 3 4 6 and a sign bit) or two's-complement
int4; x / factor and what the codes are rounded from are float32 quotients.  What a pass has appended is
returned as the values that the cache then holds.

Visibility: row r of a sequence of Sq new and Sk cached tokens (the new ones included) has position
p = Sk - Sq + r and sees the first n compressed positions, n = clamp(ceil((p + 1) / cmp), 0, ceil(Sk / cmp));
with a window w only those at n - w or later and the first `sinks`.
"""
import math

import numpy as np
import torch

own = False                     # set by the caller: True runs the library's kernels

E2M1_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
MOST_PAIRS = 64 * 128 * 44_000_000      # query heads * dim * visible (row, key) pairs, largest listed: the prefill
MOST_ENTRIES = 32 * 98_304 * 8 * 128    # cached positions * KV heads * dim, about the largest listed


# ------------------------------------------------------------------------------------------ cases
def _append(name, batch, tokens, heads_q, heads_kv, dim, rotary, kv, dtype, block_size, interleaved=False, norm=True,
            max_pos=131072, k_scale=1.0, v_scale=1.0):
    """`batch` sequences, `tokens` consecutive new tokens of each (at its end)."""
    c = dict(op="append", batch=batch, tokens=tokens, heads_q=heads_q, heads_kv=heads_kv, dim=dim, rotary=rotary, kv=kv,
             dtype=dtype, block_size=block_size, interleaved=interleaved, norm=norm, max_pos=max_pos, k_scale=k_scale,
             v_scale=v_scale)
    return dict(c, name=name) if name else c


def _attention(name, batch, s1, len_lo, len_hi, heads_q, heads_kv, dim, kv, dtype, block_size, cmp_ratio=1, window=0,
               sinks=0, news="", lens="", spare=0, short=False, lse=True, k_scale=1.0, v_scale=1.0):
    """`batch` sequences of `s1` new tokens each (BSND; `short`: some have fewer), Sk in [len_lo, len_hi]; or, with
    `news` and `lens` (comma-separated), sequences of those new and total lengths (TND, `spare` rows behind the
    last)."""
    c = dict(op="attention", batch=batch, s1=s1, len_lo=len_lo, len_hi=len_hi, heads_q=heads_q, heads_kv=heads_kv, dim=dim,
             kv=kv, dtype=dtype, block_size=block_size, cmp_ratio=cmp_ratio, window=window, sinks=sinks, news=news,
             lens=lens, spare=spare, short=short, lse=lse, k_scale=k_scale, v_scale=v_scale)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one decode step of one sequence: pure latency
        _append("append_one_token", 1, 1, 64, 8, 128, 128, "e2m1", "bf16", 64),
        # a ragged step of an int4 cache: an odd number of tokens, half of each 64-element head rotated, float16
        _append("append_ragged_f16_int4", 7, 111, 20, 5, 64, 32, "int4", "f16", 16, interleaved=True, v_scale=0.3),
        # the varlen prefill's 15360 tokens as four chunks
        _append("append_prefill", 4, 3840, 64, 8, 128, 128, "e2m1", "bf16", 128),
        # the tiny decode: one row over 256 positions
        _attention("attend_tiny", 1, 1, 256, 256, 64, 8, 128, "e2m1", "bf16", 128),
        # the page-shaped decode: 24 sequences of 4 tokens, 512 positions, some sequences with fewer tokens
        _attention("attend_page_f16_int4", 24, 4, 512, 512, 32, 4, 128, "int4", "f16", 128, short=True),
        # a dense layer's decode step: 32 sequences of 8k-32k tokens
        _attention("attend_decode", 32, 1, 8192, 32768, 64, 8, 128, "e2m1", "bf16", 64),
        # compressed keys, two tokens per sequence, 7 query heads per KV head of 64
        _attention("attend_compressed", 16, 2, 16384, 65536, 28, 4, 64, "e2m1", "bf16", 128, cmp_ratio=4, v_scale=0.5),
        # chunks of a prompt that continues: new tokens behind what is cached, odd lengths
        _attention("attend_chunks", 4, 0, 0, 0, 32, 8, 128, "e2m1", "bf16", 64, news="512,1000,33,2047",
                   lens="8192,12001,16384,30011", spare=5),
        # the varlen prefill: everything that a prompt's tokens see, the largest product
        _attention("attend_prefill", 4, 0, 0, 0, 64, 8, 128, "e2m1", "bf16", 128, news="1024,2048,4096,8192",
                   lens="1024,2048,4096,8192"),
        # a sliding-window layer's decode step with four sinks: 32 sequences of 64k-128k tokens
        _attention("window_decode", 32, 1, 65536, 131072, 64, 8, 128, "e2m1", "bf16", 64, window=4096, sinks=4),
        # a short ragged chunk with an odd window, int4, float16, heads of 64
        _attention("window_ragged_f16_int4", 3, 0, 0, 0, 15, 5, 64, "int4", "f16", 16, window=129, sinks=1,
                   news="331,1,77", lens="331,1500,2000"),
        # the varlen prefill in a sliding-window layer
        _attention("window_prefill", 4, 0, 0, 0, 64, 8, 128, "e2m1", "bf16", 128, window=1024, sinks=16,
                   news="1024,2048,4096,8192", lens="1024,2048,4096,8192"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dtype = rng.choice(("bf16", "bf16", "f16"))
    kv = rng.choice(("e2m1", "e2m1", "int4"))
    dim = rng.choice((64, 128, 128))
    block_size = rng.choice((16, 32, 48, 64, 128, 256))
    k_scale, v_scale = rng.choice(((1.0, 1.0), (0.5, 0.25), (2.0, 1.0), (1.0, 0.3)))
    heads_kv = rng.choice((1, 2, 3, 4, 5, 8, 8, 16))
    if rng.random() < 0.3:
        heads_q = heads_kv * rng.choice((0, 1, 3, 4, 7, 8))
        heads_q = heads_q if heads_q <= 64 else heads_kv * 4
        batch = rng.choice((1, 2, 3, 7, 16, 32))
        most = 15360 * (64 + 16) * 128 // ((heads_q + 2 * heads_kv) * dim * batch)
        return _append(None, batch, _log_int(rng, 1, max(1, min(most, 16384))), heads_q, heads_kv, dim,
                       rng.choice((dim, dim, dim // 2, 24)), kv, dtype, block_size, rng.random() < 0.4, rng.random() < 0.8,
                       rng.choice((40960, 131072)), k_scale, v_scale)
    group = rng.choice((1, 2, 4, 5, 7, 8, 8, 16, 32))
    heads_q = heads_kv * group if heads_kv * group <= 128 else heads_kv * 8
    window = rng.choice((0, 0, 0, _log_int(rng, 1, 8192), _log_int(rng, 16, 4096)))
    sinks = rng.choice((0, 1, 4, 16, 100)) if window else 0
    cmp_ratio = rng.choice((1, 1, 1, 2, 4))
    more = dict(cmp_ratio=cmp_ratio, window=window, sinks=sinks, lse=rng.random() < 0.7, k_scale=k_scale, v_scale=v_scale)
    while True:
        if rng.random() < 0.5:                                          # decode steps, one to a few tokens
            s1 = rng.choice((1, 1, 1, 2, 3, 4, 8))
            lo = _log_int(rng, 1, 65536)
            c = _attention(None, _log_int(rng, 1, 64), s1, lo, min(131072, lo * rng.choice((1, 2, 4))), heads_q, heads_kv,
                           dim, kv, dtype, block_size, short=s1 > 1 and rng.random() < 0.4, **more)
        else:                                                           # chunks, with or without something cached
            n = rng.choice((1, 2, 3, 5, 9))
            news = [rng.choice((1, _log_int(rng, 1, 8192), _log_int(rng, 16, 2048))) for _ in range(n)]
            old = [rng.choice((0, _log_int(rng, 1, 32768))) for _ in range(n)]
            c = _attention(None, n, 0, 0, 0, heads_q, heads_kv, dim, kv, dtype, block_size, news=",".join(map(str, news)),
                           lens=",".join(str(a + b) for a, b in zip(news, old)), spare=rng.choice((0, 0, 3)), **more)
        new, lens = _lengths(c)
        cached = int((-(-lens // cmp_ratio)).sum())
        if _pairs(c)[0] * heads_q * dim <= MOST_PAIRS and cached * heads_kv * dim <= MOST_ENTRIES:
            return c


def _lengths(case):
    """New and total tokens per sequence (from the case alone, so that work() knows them)."""
    if case["news"]:
        return tuple(np.array([int(t) for t in case[x].split(",")], np.int64) for x in ("news", "lens"))
    rng = np.random.default_rng(case["batch"] * 1000003 + case["len_lo"] * 31 + case["len_hi"])
    lens = rng.integers(case["len_lo"], case["len_hi"], size=case["batch"], endpoint=True)
    new = np.full(case["batch"], case["s1"])
    if case["short"]:
        new = rng.integers(0, case["s1"], size=case["batch"], endpoint=True)
    return new, lens


def _seen(case, new, total):
    """(first, end) of the compressed positions of each row's window, int64 [new] each."""
    end = np.clip(-(-(total - new + np.arange(new) + 1) // case["cmp_ratio"]), 0, -(-total // case["cmp_ratio"]))
    return np.maximum(end - case["window"], 0) if case["window"] else np.zeros_like(end), end


def _pairs(case):
    """Visible (row, position) pairs, and positions that some row sees."""
    pairs = distinct = 0
    for new, total in zip(*_lengths(case)):
        first, end = _seen(case, new, total)
        if new:
            pairs += int((end - first + np.minimum(first, case["sinks"])).sum())
            low = int(first[end > 0].min()) if (end > 0).any() else 0
            distinct += int(end.max()) - low + min(low, case["sinks"])
    return pairs, distinct


# ----------------------------------------------------------------------------------------- inputs
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float16


def _entry_bytes(case):
    return -(-case["heads_kv"] * (case["dim"] + case["dim"] // 8) // 16) * 16


def _pages(entries, block_size, seed):
    """block_table [B, max_blocks] for sequences of `entries` entries: pages in a random order."""
    need = [max(1, -(-int(n) // block_size)) for n in entries]
    spare = 3
    order = np.random.default_rng(seed).permutation(sum(need) + spare)
    table = np.full((len(need), max(need)), sum(need) + spare - 1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, sum(need) + spare


def _activations(shape, gen, std=1.0, channels=True):
    """Normal values; each channel with its own spread and one channel in 32 far larger."""
    x = torch.randn(shape, generator=gen, device="cuda")
    if channels:
        d = shape[-1]
        s = torch.exp(0.3 * torch.randn(d, generator=gen, device="cuda"))
        s[:: 32] *= 3.0
        x *= s
    return x.mul_(std)


def _fill_pool(case, blocks, gen):
    """A whole cache of quantised K and V.  Up to 65536 different entries, each position one of them."""
    h, d, bs = case["heads_kv"], case["dim"], case["block_size"]
    n = blocks * bs
    kinds = min(n, 65536)
    made = torch.empty((kinds, _entry_bytes(case)), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 24) // (h * d))
    for t0 in range(0, kinds, step):
        m = min(step, kinds - t0)
        k = _activations((m, h, d), gen).to(_dtype(case))
        v = _activations((m, h, d), gen, 0.5, False).to(_dtype(case))
        made[t0:t0 + m] = _pack(case, k.float(), v.float())
    if kinds < n:
        made = made[torch.randint(0, kinds, (n,), generator=gen, device="cuda")]
    return made.view(blocks, bs, -1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt, h, d, bs = _dtype(case), case["heads_kv"], case["dim"], case["block_size"]
    s = dict(case=case)
    if case["op"] == "append":
        b, n, hq, rot = case["batch"], case["tokens"], case["heads_q"], case["rotary"]
        lens = n + np.random.default_rng(int(seed)).integers(0, max(1, min(32768, case["max_pos"] - n)), size=b)
        table, blocks = _pages(lens, bs, int(seed))
        s["token_batch"] = torch.from_numpy(np.repeat(np.arange(b, dtype=np.int32), n)).cuda()
        s["token_pos"] = torch.from_numpy(np.concatenate([np.arange(m - n, m) for m in lens]).astype(np.int32)).cuda()
        s["pool"] = torch.zeros((blocks, bs, _entry_bytes(case)), dtype=torch.uint8, device="cuda")
        qkv = _activations((b * n, hq + 2 * h, d), gen).to(dt)              # the packed projection's output
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + h], qkv[:, hq + h:]
        for name in ("q_weight", "k_weight"):
            s[name] = (1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(dt) if case["norm"] else None
        s["cos_sin"] = _table(case["max_pos"], rot)
        s["q_out"] = torch.empty((b * n, hq, d), dtype=dt, device="cuda")
        s["k_out"] = torch.empty((b * n, h, d), dtype=dt, device="cuda")    # what the cache holds, read back
        s["v_out"] = torch.empty((b * n, h, d), dtype=dt, device="cuda")
        problem = dict(batch=b, max_q_tokens=n, max_seqlen_q=n, max_seqlen_k=int(lens.max()), cmp_ratio=1)
    else:
        new, lens = _lengths(case)
        comp = -(-lens // case["cmp_ratio"])
        table, blocks = _pages(comp, bs, int(seed))
        s["pool"] = _fill_pool(case, blocks, gen)
        rows = int(new.sum()) + case["spare"] if case["news"] else case["batch"] * case["s1"]
        s["first_row"] = np.cumsum(new) - new if case["news"] else np.arange(case["batch"]) * case["s1"]
        s["query"] = _activations((rows, case["heads_q"], d), gen, 1.0, False).to(dt)
        s["seq_lens_q"] = None
        if case["news"] or case["short"]:
            s["seq_lens_q"] = torch.from_numpy((np.cumsum(new) if case["news"] else new).astype(np.int32)).cuda()
        s["seq_lens_k"] = torch.from_numpy(lens.astype(np.int32)).cuda()
        s["out"] = torch.empty((rows, case["heads_q"], d), dtype=dt, device="cuda")
        s["lse"] = torch.empty((rows, case["heads_q"]), dtype=torch.float32, device="cuda") if case["lse"] else None
        problem = dict(batch=len(lens), layout_q=1 if case["news"] else 0, max_q_tokens=case["s1"], total_q_tokens=rows,
                       max_seqlen_q=int(new.max()), max_seqlen_k=int(lens.max()), cmp_ratio=case["cmp_ratio"])
    s["block_table"] = torch.from_numpy(table).cuda()
    if own:
        import sparse_attention_token_block_gb300 as Q
        s["Q"] = Q
        act = Q.ACT_BF16 if case["dtype"] == "bf16" else Q.ACT_F16
        s["p"] = Q.make_problem(num_blocks=blocks, block_size=bs, max_blocks_per_seq=table.shape[1], sparse_count=1,
                                sparse_mode=3, **problem)
        s["a"] = Q.make_attention(num_heads_q=max(case["heads_q"], h), num_heads_kv=h, head_dim=d, dtype=act,
                                  kv_dtype=Q.KV_E2M1 if case["kv"] == "e2m1" else Q.KV_INT4, k_scale=case["k_scale"],
                                  v_scale=case["v_scale"])
        if case["op"] == "append":
            s["r"] = Q.make_norm_rope(num_heads_q=case["heads_q"], num_heads_k=h, head_dim=d, rotary_dim=case["rotary"],
                                      max_positions=case["max_pos"], dtype=act, interleaved=case["interleaved"],
                                      norm=case["norm"], eps=1e-6)
        s["workspace"] = torch.zeros(64, dtype=torch.int32, device="cuda")
        Q.check(Q.workspace_init(s["workspace"]), "workspace_init")
    return s


def _table(max_pos, rot):
    """The rotation table that a server builds once (float64 angles, stored as float32)."""
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    angle = torch.arange(max_pos, dtype=torch.float64, device="cuda")[:, None] * freq[None, :]
    return torch.cat([angle.cos(), angle.sin()], 1).float()


# -------------------------------------------------------------------------------------- plain form
def _quantize(kv, x):
    """Codes (uint8, low 4 bits) and scales (float8_e4m3fn) of float32 x [..., D] in blocks of 16."""
    y = x.reshape(*x.shape[:-1], -1, 16)
    a = y.abs().amax(-1)
    top = torch.full_like(a, 6.0 if kv == "e2m1" else 7.0)      # (a tensor: a / 6.0 would multiply by 1/6)
    s = (a / top).clamp(max=448.0).to(torch.float8_e4m3fn)
    sf = s.float()[..., None]
    q = torch.where(sf > 0, y / torch.where(sf > 0, sf, torch.ones_like(sf)), torch.zeros_like(y))
    if kv == "e2m1":
        m = q.abs()
        code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0))
        code = code + 8 * (q < 0).to(torch.uint8)
    else:
        code = (torch.round(q).clamp(-7, 7).to(torch.int8) & 15).to(torch.uint8)
    return code.reshape(x.shape), s


def _pack(case, k, v):
    """Cache entries uint8 [T, entry_bytes] of float32 k, v [T, H, D]."""
    gk, gv = torch.full_like(k, case["k_scale"]), torch.full_like(v, case["v_scale"])       # (true divisions)
    (kc, ks), (vc, vs) = _quantize(case["kv"], k / gk), _quantize(case["kv"], v / gv)
    e = torch.cat([kc[..., 0::2] | (kc[..., 1::2] << 4), vc[..., 0::2] | (vc[..., 1::2] << 4), ks.view(torch.uint8),
                   vs.view(torch.uint8)], -1).flatten(1)
    return torch.nn.functional.pad(e, (0, _entry_bytes(case) - e.shape[1]))


def _unpack(case, entries):
    """float32 K and V [T, H, D] of entries uint8 [T, entry_bytes]."""
    h, d = case["heads_kv"], case["dim"]
    e = entries[:, :h * (d + d // 8)].unflatten(-1, (h, d + d // 8))
    code = torch.stack([e[..., :d] & 15, e[..., :d] >> 4], -1).flatten(-2).to(torch.int32)      # K's, then V's
    if case["kv"] == "e2m1":
        val = torch.tensor(E2M1_GRID + tuple(-x for x in E2M1_GRID), device=e.device)[code]
    else:
        val = torch.where(code < 8, code, code - 16).float()
    scale = e[..., d:].contiguous().view(torch.float8_e4m3fn).float()
    val = (val.unflatten(-1, (d // 8, 16)) * scale[..., None]).flatten(-2)
    return val[..., :d] * case["k_scale"], val[..., d:] * case["v_scale"]


def _plain_append(s):
    case = s["case"]
    rot, half = case["rotary"], case["rotary"] // 2
    cs = s["cos_sin"][s["token_pos"].long()][:, None, :]
    cos, sin = cs[..., :half], cs[..., half:]
    first, second = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (slice(0, half), slice(half, rot))

    def turned(x, w):
        y = x.float()
        if case["norm"]:
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w.float()
        z = y.clone()
        z[..., first] = y[..., first] * cos - y[..., second] * sin
        z[..., second] = y[..., second] * cos + y[..., first] * sin
        return z

    pos, bs = s["token_pos"].long(), case["block_size"]
    page, slot = s["block_table"][s["token_batch"].long(), pos // bs].long(), pos % bs
    s["pool"][page, slot] = _pack(case, turned(s["k"], s["k_weight"]), s["v"].float())
    k, v = _unpack(case, s["pool"][page, slot])
    return {"q": turned(s["q"], s["q_weight"]).to(_dtype(case)), "k": k.to(_dtype(case)), "v": v.to(_dtype(case))}


def _spans(case, limit):
    """(sequence, first row, end row, first window position, end position) of blocks of rows of at most `limit` logits."""
    for b, (new, total) in enumerate(zip(*_lengths(case))):
        r = 0
        while r < new:
            first, end = _seen(case, new, total)
            if case["window"]:                                          # m rows see at most window + m positions
                w = case["window"]
                m = int((math.sqrt(w * w + 4 * limit / case["heads_q"]) - w) / 2)
            else:
                m = limit // (max(1, int(end.max())) * case["heads_q"])
            m = int(min(new - r, max(1, m)))
            yield b, r, r + m, int(first[r]), int(end[r + m - 1])
            r += m


def _plain_attention(s):
    case = s["case"]
    h, d, hq, bs = case["heads_kv"], case["dim"], case["heads_q"], case["block_size"]
    out = torch.zeros_like(s["out"])
    lse = torch.full(s["out"].shape[:2], -math.inf, device="cuda")
    lengths = _lengths(case)
    for b, r0, r1, lo, hi in _spans(case, 1 << 28):
        pos = torch.arange(lo, hi, device="cuda")
        if lo > 0:
            pos = torch.cat([torch.arange(0, min(lo, case["sinks"]), device="cuda"), pos])
        k, v = _unpack(case, s["pool"][s["block_table"][b, pos // bs].long(), pos % bs])
        at = int(s["first_row"][b]) + r0
        q = s["query"][at:at + r1 - r0].float().view(r1 - r0, h, hq // h, d)
        z = torch.einsum("rhgd,nhd->hgrn", q, k) * (1.0 / math.sqrt(d))
        new, total = int(lengths[0][b]), int(lengths[1][b])
        p = total - new + torch.arange(r0, r1, device="cuda")[:, None]      # the rows' positions
        end = ((p + case["cmp_ratio"]) // case["cmp_ratio"]).clamp(0, -(-total // case["cmp_ratio"]))
        seen = pos < end
        if case["window"]:
            seen &= (pos >= end - case["window"]) | (pos < case["sinks"])
        z = z.masked_fill(~seen, -math.inf)
        top = z.amax(-1, keepdim=True) if pos.numel() else z.new_full(z.shape[:-1] + (1,), -math.inf)
        top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
        z = torch.exp(z - top)
        sums = z.sum(-1, keepdim=True)
        o = torch.einsum("hgrn,nhd->rhgd", z / torch.where(sums > 0, sums, torch.ones_like(sums)), v)
        out[at:at + r1 - r0] = o.reshape(r1 - r0, hq, d).to(out.dtype)
        lse[at:at + r1 - r0] = (top + torch.log(sums)).flatten(0, 1)[..., 0].t()
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}


# ------------------------------------------------------------------------------------------- a pass
def run(s):
    op = s["case"]["op"]
    if not own:
        return _plain_append(s) if op == "append" else _plain_attention(s)
    Q = s["Q"]
    if op == "attention":
        Q.check(Q.paged_attention(s["p"], s["a"], s["query"], s["seq_lens_q"], s["seq_lens_k"], s["block_table"], s["pool"],
                                  s["out"], s["lse"], s["workspace"], window=s["case"]["window"], sinks=s["case"]["sinks"]),
                "paged_attention")
        return {"out": s["out"], "lse": s["lse"]} if s["lse"] is not None else {"out": s["out"]}
    Q.check(Q.kv_append(s["p"], s["a"], s["r"], s["q"], s["k"], s["v"], s["q_weight"], s["k_weight"], s["token_pos"],
                        s["cos_sin"], s["token_batch"], s["token_pos"], s["block_table"], s["q_out"], s["pool"],
                        s["workspace"]), "kv_append")
    Q.check(Q.kv_read(s["p"], s["a"], s["token_batch"], s["token_pos"], s["block_table"], s["pool"], s["k_out"],
                      s["v_out"], s["workspace"]), "kv_read")
    return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}


def work(case):
    entry, d = _entry_bytes(case), case["dim"]
    if case["op"] == "append":
        # activations in and out, the entries written and read back, a table row and three places a token
        n = case["batch"] * case["tokens"]
        values = n * (case["heads_q"] + 2 * case["heads_kv"]) * d
        return {"bytes": 4 * values + 2 * n * entry + n * (4 * case["rotary"] + 8), "flops": 12 * values}
    pairs, distinct = _pairs(case)
    new, lens = _lengths(case)
    rows = int(new.sum()) + case["spare"] if case["news"] else case["batch"] * case["s1"]
    seen = -(-distinct // case["block_size"])
    return {"bytes": distinct * entry + 4 * seen + rows * case["heads_q"] * (4 * d + (4 if case["lse"] else 0)),
            "flops": 4 * pairs * case["heads_q"] * d}


# ------------------------------------------------------------------------------- the same in 64 bits
def _exact_e4m3(a):
    """Nearest float8_e4m3fn (ties to even) of a >= 0, at most 448, as float64."""
    a = a.clamp(max=448.0)
    b = a.clamp(min=2.0 ** -6)
    step = b / torch.frexp(b)[0] / 16                           # b / its mantissa: an exact power of two
    return (torch.round(a / step) * step).clamp(max=448.0)


def _f32(x):
    return x.float().double()


def _exact_values(kv, x):
    """The values that x [..., D] (float64) has in the cache; the format's quotients are float32 numbers."""
    y = _f32(x).unflatten(-1, (-1, 16))
    top = 6.0 if kv == "e2m1" else 7.0
    a = y.abs().amax(-1, keepdim=True)
    s = _exact_e4m3(_f32(a / torch.full_like(a, top)))          # (a true division: ties stay ties)
    q = _f32(y / torch.where(s == 0, torch.full_like(s, math.inf), s))
    if kv == "e2m1":
        b = q.abs().clamp(min=1.0)
        step = b / torch.frexp(b)[0] / 4
        c = torch.round(q / step) * step
    else:
        c = torch.round(q)
    return (c.clamp(-top, top) * s).flatten(-2)


def _exact_entries(case, raw):
    """float64 K and V [H, T, D] of raw entries [T, entry_bytes], byte by byte."""
    h, d = case["heads_kv"], case["dim"]
    byte = torch.arange(256, device="cuda")
    if case["kv"] == "e2m1":
        nib = torch.tensor([(1 - 2 * (c >> 3)) * ((c & 7) * 0.5 if c & 7 < 2 else (1 + (c & 1) / 2) * 2.0 ** (((c >> 1) & 3) - 1))
                            for c in range(16)], dtype=torch.float64, device="cuda")
        nib[1], nib[9] = 0.5, -0.5
    else:
        nib = torch.tensor([c - 16 * (c >> 3) for c in range(16)], dtype=torch.float64, device="cuda")
    pairs = torch.stack([nib[byte & 15], nib[byte >> 4]], 1)            # [256, 2]
    scale = torch.tensor([(1 - 2 * (c >> 7)) * ((8 + (c & 7)) * 2.0 ** (((c >> 3) & 15) - 10) if c & 120 else (c & 7) * 2.0 ** -9)
                          for c in range(256)], dtype=torch.float64, device="cuda")
    unit = d + d // 8
    e = raw[:, :h * unit].reshape(-1, h, unit).transpose(0, 1).long()
    return [pairs[e[..., at:at + d // 2]].flatten(-2) * scale[e[..., sat:sat + d // 16]].repeat_interleave(16, -1) * g
            for at, sat, g in ((0, d, case["k_scale"]), (d // 2, d + d // 16, case["v_scale"]))]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        table = s["cos_sin"].double().index_select(0, s["token_pos"].long())
        rot = case["rotary"]
        ang = torch.complex(table[:, :rot // 2], table[:, rot // 2:])[:, None, :]
        res = {}
        for name in ("q", "k"):
            x = s[name].double()
            if case["norm"]:
                x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / case["dim"] + 1e-6) * s[name + "_weight"].double()
            a, rest = x[..., :rot], x[..., rot:]
            if case["interleaved"]:
                a = torch.view_as_real(torch.complex(a[..., 0::2].contiguous(), a[..., 1::2].contiguous()) * ang).flatten(-2)
            else:
                w = torch.complex(a[..., :rot // 2].contiguous(), a[..., rot // 2:].contiguous()) * ang
                a = torch.cat([w.real, w.imag], -1)
            res[name] = torch.cat([a, rest], -1)
        gk, gv = float(np.float32(case["k_scale"])), float(np.float32(case["v_scale"]))
        return {"q": res["q"], "k": _exact_values(case["kv"], res["k"] / gk) * gk,
                "v": _exact_values(case["kv"], s["v"].double() / gv) * gv}
    h, d, hq, bs, cmp = case["heads_kv"], case["dim"], case["heads_q"], case["block_size"], case["cmp_ratio"]
    flat, table = s["pool"].reshape(-1, s["pool"].shape[-1]), s["block_table"].long()
    rows = s["query"].shape[0]
    out = torch.zeros((rows, hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((rows, hq), -math.inf, dtype=torch.float64, device="cuda")
    news, lens = _lengths(case)
    for b, r0, r1, lo, hi in _spans(case, 1 << 26):
        low = min(lo, case["sinks"])
        j = torch.arange(low + hi - lo, device="cuda")
        j = torch.where(j < low, j, j - low + lo)
        k, v = _exact_entries(case, flat[table[b][j // bs] * bs + j % bs])              # [h, n, d]
        at = int(s["first_row"][b]) + r0
        q = s["query"][at:at + r1 - r0].double().reshape(r1 - r0, h, hq // h, d).permute(1, 2, 0, 3).flatten(1, 2)
        z = (q @ k.transpose(1, 2) / math.sqrt(d)).unflatten(1, (hq // h, r1 - r0))     # [h, g, r, n]
        last = int(lens[b] - news[b]) + torch.arange(r0, r1, device="cuda")             # a key of original tokens
        n = torch.where(last >= 0, last // cmp + 1, 0)[:, None]                         # j cmp <= last is visible
        hidden = (j >= n) | ((j < n - case["window"]) & (j >= case["sinks"])) if case["window"] else j >= n
        z = torch.where(hidden, torch.full_like(z, -math.inf), z)
        total = torch.logsumexp(z, -1) if j.numel() else z.new_full(z.shape[:-1], -math.inf)
        w = torch.where(torch.isfinite(total)[..., None], torch.exp(z - total[..., None]), torch.zeros_like(z))
        o = (w.flatten(1, 2) @ v).unflatten(1, (hq // h, r1 - r0))
        out[at:at + r1 - r0] = o.permute(2, 0, 1, 3).flatten(1, 2)
        lse[at:at + r1 - r0] = total.flatten(0, 1).t()
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}
