"""Workloads of the attention-side operators: per-head norm with rotation, the 4-bit paged KV cache
(write and read back), and sparse attention over the entries an index list names.

Every case has a plain form (elementary torch operations, float32) and, with ``own`` set, the calls
that a user makes of the library.  ``listed()`` gives the named cases, ``draw(rng)`` one more of the
same ranges, ``prepare`` the inputs, ``run`` one pass, ``exact`` the same outputs in 64 bits.

Cache format (both forms keep the same bytes): the entry of a token holds, for each KV head, D/2
bytes of K codes, D/2 bytes of V codes, D/16 bytes of K scales and D/16 bytes of V scales, padded to
16 bytes; element 2i of a vector is the low nibble of byte i; scales are float8_e4m3fn, one per 16
elements; codes are E2M1 (values 0 .5 1 1.5 2 3 4 6 and a sign bit) or two's-complement int4.
"""
import math

import numpy as np
import torch

own = False                     # set by the caller: True runs the library's kernels

E2M1_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
MAX_ATTENTION_WORK = 7168 * 2048 * 64 * 128         # rows * list * query heads * dim, largest listed


# ------------------------------------------------------------------------------------------ cases
def _norm_rope(name, tokens, heads_q, heads_kv, dim, rotary, dtype, interleaved=False, norm=True,
               max_pos=131072, consecutive=False):
    c = dict(op="norm_rope", tokens=tokens, heads_q=heads_q, heads_kv=heads_kv, dim=dim, rotary=rotary,
             dtype=dtype, interleaved=interleaved, norm=norm, max_pos=max_pos, consecutive=consecutive)
    return dict(c, name=name) if name else c


def _cache(name, op, batch, tokens, heads_kv, dim, kv, dtype, block_size, k_scale=1.0, v_scale=1.0):
    """`batch` sequences, `tokens` consecutive entries of each (at its end)."""
    c = dict(op=op, batch=batch, tokens=tokens, heads_kv=heads_kv, dim=dim, kv=kv, dtype=dtype,
             block_size=block_size, k_scale=k_scale, v_scale=v_scale)
    return dict(c, name=name) if name else c


def _attention(name, batch, s1, len_lo, len_hi, k, heads_q, heads_kv, dim, kv, dtype, block_size, cmp_ratio=1,
               lens="", empty_every=0, lse=True, k_scale=1.0, v_scale=1.0):
    """Decode (`s1` query tokens per sequence, S_k in [len_lo, len_hi]) or, with `lens`, a causal
    prefill of sequences of those lengths (comma-separated, TND)."""
    c = dict(op="attention", batch=batch, s1=s1, len_lo=len_lo, len_hi=len_hi, k=k, heads_q=heads_q,
             heads_kv=heads_kv, dim=dim, kv=kv, dtype=dtype, block_size=block_size, cmp_ratio=cmp_ratio,
             lens=lens, empty_every=empty_every, lse=lse, k_scale=k_scale, v_scale=v_scale)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one decode step of one sequence: pure latency
        _norm_rope("norm_rope_one_token", 1, 64, 8, 128, 128, "bf16"),
        # an odd number of tokens, half of each 64-element head rotated in interleaved pairs, float16
        _norm_rope("norm_rope_ragged_f16", 777, 20, 5, 64, 32, "f16", interleaved=True),
        # the varlen prefill's 15360 tokens
        _norm_rope("norm_rope_prefill", 15360, 64, 8, 128, 128, "bf16", consecutive=True),
        # one decode step of 32 sequences appends one token each, then reads it back
        _cache("write_decode", "kv_write", 32, 1, 8, 128, "e2m1", "bf16", 64),
        # a prefill chunk written to the cache and read back as the values the cache holds
        _cache("write_prefill", "kv_write", 4, 3840, 8, 128, "e2m1", "bf16", 128, v_scale=0.25),
        # a short odd tail of an int4 cache with 64-element heads
        _cache("read_ragged_int4", "kv_read", 3, 331, 5, 64, "int4", "f16", 16),
        # long cached prefixes read back for a dense pass
        _cache("read_prefix", "kv_read", 8, 8192, 8, 128, "e2m1", "bf16", 64),
        # the tiny decode: one row, 64 entries
        _attention("attention_tiny", 1, 1, 256, 256, 64, 64, 8, 128, "e2m1", "bf16", 128),
        # the page-shaped decode: 24 sequences, 4 tokens each, lists as long as the cache
        _attention("attention_page", 24, 4, 512, 512, 512, 32, 4, 128, "int4", "f16", 128),
        # the long decode: 32 sequences of 8k-32k keys, 2048 selected, a padding row now and then
        _attention("attention_long_decode", 32, 1, 8192, 32768, 2048, 64, 8, 128, "e2m1", "bf16", 64,
                   empty_every=16),
        # the compressed decode: two tokens per sequence, keys compressed 4x, 7 query heads per KV head
        _attention("attention_compressed", 16, 2, 16384, 65536, 2048, 28, 4, 64, "e2m1", "bf16", 128, cmp_ratio=4,
                   v_scale=0.5),
        # three sequences of the varlen prefill: 7168 causal rows, up to 2048 selected each
        _attention("attention_prefill", 3, 0, 0, 0, 2048, 64, 8, 128, "e2m1", "bf16", 128,
                   lens="1024,2048,4096"),
    ]


def draw(rng):
    while True:
        case = _draw(rng)
        row = case["dim"] * case.get("heads_q", case["heads_kv"])
        if 3072 not in (row, case["dim"] * case["heads_kv"], case["batch"] * case.get("tokens", 1) if "batch" in case else 0):
            return case


def _draw(rng):
    def log_int(lo, hi):
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        return v + 1 if v == 3072 else v

    op = rng.choice(("norm_rope", "kv_write", "kv_read", "attention", "attention", "attention"))
    dtype = rng.choice(("bf16", "bf16", "f16"))
    if op == "norm_rope":
        dim = rng.choice((64, 128, 128, 256))
        heads_kv = rng.choice((1, 2, 3, 5, 8))
        heads_q = heads_kv * rng.choice((1, 3, 4, 7, 8))
        rotary = rng.choice((dim, dim, dim // 2, 24))
        return _norm_rope(None, log_int(1, 15360 * 8 * 128 // (dim * heads_kv)) if heads_q <= 64 else log_int(1, 8192),
                          heads_q, heads_kv, dim, rotary, dtype, rng.random() < 0.4, rng.random() < 0.8,
                          rng.choice((4096, 40960, 131072)), rng.random() < 0.5)
    kv = rng.choice(("e2m1", "int4"))
    dim = rng.choice((64, 128, 128))
    block_size = rng.choice((16, 32, 48, 64, 128, 256))
    scales = rng.choice(((1.0, 1.0), (0.5, 0.25), (2.0, 1.0)))
    if op != "attention":
        heads_kv = rng.choice((1, 2, 3, 5, 8, 16))
        batch = rng.choice((1, 2, 3, 7, 16, 32))
        most = 65536 * 8 * 128 // (2 * heads_kv * dim * batch)
        return _cache(None, op, batch, log_int(1, min(most, 16384)), heads_kv, dim, kv, dtype, block_size, *scales)
    heads_kv = rng.choice((1, 2, 3, 4, 5, 8, 8, 16))
    group = rng.choice((1, 2, 4, 5, 7, 8, 8, 16, 32))
    heads_q = heads_kv * group
    if heads_q > 128:
        heads_q = heads_kv * 8
    k = log_int(1, 2048)
    empty = rng.choice((0, 0, 0, 2, 5))
    if rng.random() < 0.3:                                   # a prefill
        lens = [log_int(1, 4096) for _ in range(rng.choice((1, 2, 3, 5)))]
        while sum(lens) * k * heads_q * dim > MAX_ATTENTION_WORK:
            lens = [max(1, n // 2) for n in lens]
        return _attention(None, len(lens), 0, 0, 0, k, heads_q, heads_kv, dim, kv, dtype, block_size,
                          lens=",".join(str(n) for n in lens), empty_every=empty, lse=rng.random() < 0.7,
                          k_scale=scales[0], v_scale=scales[1])
    lo = log_int(1, 16384)
    return _attention(None, log_int(1, 64), rng.choice((1, 1, 1, 2, 3, 4)), lo, min(65536, lo * rng.choice((1, 2, 4))), k,
                      heads_q, heads_kv, dim, kv, dtype, block_size, cmp_ratio=rng.choice((1, 1, 1, 2, 4)),
                      empty_every=empty, lse=rng.random() < 0.7, k_scale=scales[0], v_scale=scales[1])


# ----------------------------------------------------------------------------------------- inputs
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float16


def _entry_bytes(case):
    return -(-case["heads_kv"] * (case["dim"] + case["dim"] // 8) // 16) * 16


def _key_lens(case):
    """Original key tokens per sequence (drawn from the case alone, so that work() knows them)."""
    if case["lens"]:
        return np.array([int(t) for t in case["lens"].split(",")], np.int32)
    rng = np.random.default_rng(case["batch"] * 1000003 + case["len_lo"] * 31 + case["len_hi"])
    return rng.integers(case["len_lo"], case["len_hi"], size=case["batch"], endpoint=True).astype(np.int32)


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
    """A whole cache of quantised K and V, made page range by page range."""
    h, d, bs = case["heads_kv"], case["dim"], case["block_size"]
    pool = torch.empty((blocks, bs, _entry_bytes(case)), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 24) // (bs * h * d))
    for b0 in range(0, blocks, step):
        n = min(step, blocks - b0)
        k = _activations((n * bs, h, d), gen).to(_dtype(case))
        v = _activations((n * bs, h, d), gen, 0.5, False).to(_dtype(case))
        pool[b0:b0 + n] = _pack(case, k, v).view(n, bs, -1)
    return pool


def _index_lists(case, lens, gen):
    """What the indexer leaves: per row, distinct visible positions in score order, -1 at the end."""
    k = case["k"]
    comp = [-(-int(n) // case["cmp_ratio"]) for n in lens]
    parts = []
    for b, lc in enumerate(comp):
        rows = int(lens[b]) if case["lens"] else case["s1"]
        for r0 in range(0, rows, 1024):
            n = min(1024, rows - r0)
            key = torch.rand((n, lc), generator=gen, device="cuda")
            key += torch.linspace(0, 0.5, lc, device="cuda")         # later positions more often
            pos = torch.arange(lc, device="cuda")
            if case["lens"]:
                last = torch.arange(r0, r0 + n, device="cuda")
            else:                                                    # right-aligned query tokens
                last = (int(lens[b]) - rows + torch.arange(r0, r0 + n, device="cuda")) // case["cmp_ratio"]
            key = torch.where(pos[None, :] <= last[:, None], key, torch.full_like(key, -1.0))
            top, idx = torch.topk(key, min(k, lc), dim=1)
            out = torch.full((n, k), -1, dtype=torch.int32, device="cuda")
            out[:, :idx.shape[1]] = torch.where(top >= 0, idx, torch.full_like(idx, -1)).int()
            parts.append(out)
    lists = torch.cat(parts)
    if case["empty_every"]:
        lists[case["empty_every"] - 1::case["empty_every"]] = -1
    return lists


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = _dtype(case)
    s = dict(case=case)
    if case["op"] == "norm_rope":
        t, hq, hk, d, rot = case["tokens"], case["heads_q"], case["heads_kv"], case["dim"], case["rotary"]
        qkv = _activations((t, hq + 2 * hk, d), gen).to(dt)           # the packed projection's output
        s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hk]
        s["q_weight"] = (1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(dt) if case["norm"] else None
        s["k_weight"] = (1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(dt) if case["norm"] else None
        s["cos_sin"] = _table(case["max_pos"], rot)
        if case["consecutive"]:
            first = torch.randint(0, max(1, case["max_pos"] - t), (1,), generator=gen, device="cuda")
            s["positions"] = ((first + torch.arange(t, device="cuda")) % case["max_pos"]).int()
        else:
            s["positions"] = torch.randint(0, case["max_pos"], (t,), generator=gen, device="cuda").int()
        s["q_out"] = torch.empty((t, hq, d), dtype=dt, device="cuda")
        s["k_out"] = torch.empty((t, hk, d), dtype=dt, device="cuda")
        if own:
            import sparse_attention_token_block_gb300 as Q
            s["Q"] = Q
            s["r"] = Q.make_norm_rope(num_heads_q=hq, num_heads_k=hk, head_dim=d, rotary_dim=rot,
                                      max_positions=case["max_pos"], dtype=_own_dtype(Q, case),
                                      interleaved=case["interleaved"], norm=case["norm"], eps=1e-6)
        return s

    h, d, bs = case["heads_kv"], case["dim"], case["block_size"]
    if case["op"] in ("kv_write", "kv_read"):
        b, n = case["batch"], case["tokens"]
        rng = np.random.default_rng(int(seed))
        lens = n + rng.integers(0, 2 * bs, size=b)                    # entries held, the last n are dealt with
        table, blocks = _pages(lens, bs, int(seed))
        s["token_batch"] = torch.from_numpy(np.repeat(np.arange(b, dtype=np.int32), n)).cuda()
        s["token_pos"] = torch.from_numpy(np.concatenate([np.arange(m - n, m) for m in lens]).astype(np.int32)).cuda()
        s["pool"] = _fill_pool(case, blocks, gen)
        if case["op"] == "kv_write":
            qkv = _activations((b * n, 3 * h, d), gen).to(dt)
            s["k"], s["v"] = qkv[:, h:2 * h], qkv[:, 2 * h:]
        s["k_out"] = torch.empty((b * n, h, d), dtype=dt, device="cuda")
        s["v_out"] = torch.empty((b * n, h, d), dtype=dt, device="cuda")
        problem = dict(batch=b, max_q_tokens=1, sparse_count=1, sparse_mode=0, cmp_ratio=1, max_seqlen_q=1,
                       max_seqlen_k=int(lens.max()))
    else:
        lens = _key_lens(case)
        comp = -(-lens.astype(np.int64) // case["cmp_ratio"])
        table, blocks = _pages(comp, bs, int(seed))
        s["pool"] = _fill_pool(case, blocks, gen)
        s["indices"] = _index_lists(case, lens, gen)
        rows = s["indices"].shape[0]
        s["query"] = _activations((rows, case["heads_q"], d), gen, 1.0, False).to(dt)
        s["seq_lens_k"] = torch.from_numpy(lens).cuda()
        s["seq_lens_q"] = torch.from_numpy(np.cumsum(lens, dtype=np.int32)).cuda() if case["lens"] else None
        s["row_batch"] = torch.from_numpy(np.repeat(np.arange(len(lens)), lens if case["lens"] else case["s1"])).cuda()
        s["out"] = torch.empty((rows, case["heads_q"], d), dtype=dt, device="cuda")
        s["lse"] = torch.empty((rows, case["heads_q"]), dtype=torch.float32, device="cuda") if case["lse"] else None
        problem = dict(batch=len(lens), layout_q=1 if case["lens"] else 0, max_q_tokens=case["s1"], total_q_tokens=rows,
                       sparse_count=case["k"], sparse_mode=3, cmp_ratio=case["cmp_ratio"],
                       max_seqlen_q=int(lens.max()) if case["lens"] else case["s1"], max_seqlen_k=int(lens.max()))
    s["block_table"] = torch.from_numpy(table).cuda()
    if own:
        import sparse_attention_token_block_gb300 as Q
        s["Q"] = Q
        s["p"] = Q.make_problem(num_blocks=blocks, block_size=bs, max_blocks_per_seq=table.shape[1], **problem)
        s["a"] = Q.make_attention(num_heads_q=case.get("heads_q", h), num_heads_kv=h, head_dim=d,
                                  dtype=_own_dtype(Q, case), kv_dtype=Q.KV_E2M1 if case["kv"] == "e2m1" else Q.KV_INT4,
                                  k_scale=case["k_scale"], v_scale=case["v_scale"])
        s["workspace"] = torch.zeros(64, dtype=torch.int32, device="cuda")
        Q.check(Q.workspace_init(s["workspace"]), "workspace_init")
    return s


def _table(max_pos, rot):
    """The rotation table that a server builds once (float64 angles, stored as float32)."""
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    angle = torch.arange(max_pos, dtype=torch.float64, device="cuda")[:, None] * freq[None, :]
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def _own_dtype(Q, case):
    return Q.ACT_BF16 if case["dtype"] == "bf16" else Q.ACT_F16


# -------------------------------------------------------------------------------------- plain form
def _quantize(kv, x):
    """Codes (uint8, low 4 bits) and scales (float8_e4m3fn) of x [..., D] in blocks of 16."""
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
    """Cache entries uint8 [T, entry_bytes] of k, v [T, H, D]."""
    parts_code, parts_scale = [], []
    for x, g in ((k, case["k_scale"]), (v, case["v_scale"])):
        code, s = _quantize(case["kv"], x.float() / g)
        parts_code.append(code[..., 0::2] | (code[..., 1::2] << 4))
        parts_scale.append(s.view(torch.uint8))
    e = torch.cat(parts_code + parts_scale, -1).flatten(1)
    pad = _entry_bytes(case) - e.shape[1]
    return torch.nn.functional.pad(e, (0, pad)) if pad else e


def _unpack(case, entries):
    """float32 K and V [..., H, D] of entries uint8 [..., entry_bytes]."""
    h, d = case["heads_kv"], case["dim"]
    e = entries[..., :h * (d + d // 8)].unflatten(-1, (h, d + d // 8))
    out = []
    for at, sc, g in ((0, d, case["k_scale"]), (d // 2, d + d // 16, case["v_scale"])):
        b = e[..., at:at + d // 2]
        code = torch.stack([b & 15, b >> 4], -1).flatten(-2).to(torch.int32)
        if case["kv"] == "e2m1":
            grid = torch.tensor(E2M1_GRID + tuple(-x for x in E2M1_GRID), device=e.device)
            val = grid[code]
        else:
            val = torch.where(code < 8, code, code - 16).float()
        s = e[..., sc:sc + d // 16].contiguous().view(torch.float8_e4m3fn).float()
        out.append((val.unflatten(-1, (d // 16, 16)) * s[..., None]).flatten(-2) * g)
    return out


def _slots(s, batch, pos):
    """(page, slot) of positions through the block_table."""
    bs = s["case"]["block_size"]
    return s["block_table"][batch.long(), (pos // bs).long()].long(), (pos % bs).long()


def _plain_norm_rope(s):
    case = s["case"]
    rot, half = case["rotary"], case["rotary"] // 2
    cs = s["cos_sin"][s["positions"].long()][:, None, :]
    cos, sin = cs[..., :half], cs[..., half:]
    res = []
    for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        y = x.float()
        if case["norm"]:
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w.float()
        z = y.clone()
        first, second = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (slice(0, half), slice(half, rot))
        z[..., first] = y[..., first] * cos - y[..., second] * sin
        z[..., second] = y[..., second] * cos + y[..., first] * sin
        res.append(z.to(x.dtype))
    return {"q": res[0], "k": res[1]}


def _plain_cache(s):
    case = s["case"]
    page, slot = _slots(s, s["token_batch"], s["token_pos"])
    if case["op"] == "kv_write":
        s["pool"][page, slot] = _pack(case, s["k"], s["v"])
    k, v = _unpack(case, s["pool"][page, slot])
    return {"k": k.to(_dtype(case)), "v": v.to(_dtype(case))}


def _plain_attention(s):
    case = s["case"]
    h, d, n = case["heads_kv"], case["dim"], case["k"]
    g = case["heads_q"] // h
    rows = s["indices"].shape[0]
    outs, lses = [], []
    step = max(1, (1 << 28) // (n * h * d))
    for r0 in range(0, rows, step):
        idx = s["indices"][r0:r0 + step]
        ok = idx >= 0
        page, slot = _slots(s, s["row_batch"][r0:r0 + step, None].expand_as(idx), idx.clamp(min=0))
        k, v = _unpack(case, s["pool"][page, slot])                     # [r, n, h, d]
        q = s["query"][r0:r0 + step].float().view(-1, h, g, d)
        z = torch.einsum("rhgd,rnhd->rhgn", q, k) * (1.0 / math.sqrt(d))
        z = z.masked_fill(~ok[:, None, None, :], -math.inf)
        top = z.amax(-1, keepdim=True)
        top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
        e = torch.exp(z - top)
        total = e.sum(-1, keepdim=True)
        o = torch.einsum("rhgn,rnhd->rhgd", e, v) / torch.where(total > 0, total, torch.ones_like(total))
        outs.append(o.reshape(-1, h * g, d).to(_dtype(case)))
        lses.append((top + torch.log(total)).reshape(-1, h * g))
    out = {"out": torch.cat(outs)}
    if case["lse"]:
        out["lse"] = torch.cat(lses)
    return out


# ------------------------------------------------------------------------------------------- a pass
def run(s):
    op = s["case"]["op"]
    if not own:
        return {"norm_rope": _plain_norm_rope, "kv_write": _plain_cache, "kv_read": _plain_cache,
                "attention": _plain_attention}[op](s)
    Q = s["Q"]
    if op == "norm_rope":
        Q.check(Q.norm_rope(s["r"], s["q"], s["k"], s["q_weight"], s["k_weight"], s["positions"], s["cos_sin"],
                            s["q_out"], s["k_out"]), "norm_rope")
        return {"q": s["q_out"], "k": s["k_out"]}
    if op == "attention":
        Q.check(Q.sparse_attention(s["p"], s["a"], s["query"], s["seq_lens_q"], s["seq_lens_k"], s["block_table"],
                                   s["indices"], s["pool"], s["out"], s["lse"], s["workspace"]), "sparse_attention")
        return {"out": s["out"], "lse": s["lse"]} if s["lse"] is not None else {"out": s["out"]}
    if op == "kv_write":
        Q.check(Q.kv_write(s["p"], s["a"], s["k"], s["v"], s["token_batch"], s["token_pos"], s["block_table"],
                           s["pool"], s["workspace"]), "kv_write")
    Q.check(Q.kv_read(s["p"], s["a"], s["token_batch"], s["token_pos"], s["block_table"], s["pool"], s["k_out"],
                      s["v_out"], s["workspace"]), "kv_read")
    return {"k": s["k_out"], "v": s["v_out"]}


def work(case):
    if case["op"] == "norm_rope":
        n = case["tokens"] * (case["heads_q"] + case["heads_kv"]) * case["dim"]
        return {"bytes": 4 * n + case["tokens"] * (4 + 4 * case["rotary"]) + 4 * case["dim"], "flops": 8 * n}
    entry = _entry_bytes(case)
    if case["op"] != "attention":
        n = case["batch"] * case["tokens"]
        values = 2 * n * case["heads_kv"] * case["dim"]
        # a write pass writes the entries and reads them back; the values go in (write) and out
        both = case["op"] == "kv_write"
        return {"bytes": n * (entry * (2 if both else 1) + 8) + values * (4 if both else 2), "flops": 4 * values}
    lens = _key_lens(case)
    comp = -(-lens.astype(np.int64) // case["cmp_ratio"])
    rows = lens if case["lens"] else np.full(len(lens), case["s1"])
    listed_n = 0
    distinct = 0
    for n, lc, r in zip(lens, comp, rows):
        if case["lens"]:
            per_row = int(np.minimum(np.arange(1, n + 1), case["k"]).sum())
        else:
            per_row = int(r) * int(min(case["k"], lc))
        listed_n += per_row
        distinct += min(int(lc), per_row)
    total = int(rows.sum())
    return {"bytes": distinct * entry + 4 * total * case["k"] + total * case["heads_q"] * (4 * case["dim"] + (4 if case["lse"] else 0)),
            "flops": 4 * listed_n * case["heads_q"] * case["dim"]}


# ------------------------------------------------------------------------------- the same in 64 bits
def _exact_e4m3(a):
    """Nearest float8_e4m3fn (ties to even) of a >= 0, at most 448, as float64."""
    a = a.clamp(max=448.0)
    b = a.clamp(min=2.0 ** -6)
    step = b / torch.frexp(b)[0] / 16                           # b / its mantissa: an exact power of two
    return (torch.round(a / step) * step).clamp(max=448.0)


def _exact_values(kv, x):
    """The values that x [..., D] (float64) has in the cache."""
    y = x.unflatten(-1, (-1, 16))
    top = 6.0 if kv == "e2m1" else 7.0
    a = y.abs().amax(-1, keepdim=True)
    s = _exact_e4m3(a / torch.full_like(a, top))                # (a true division: ties stay ties)
    q = y / torch.where(s == 0, torch.full_like(s, math.inf), s)
    if kv == "e2m1":
        b = q.abs().clamp(min=1.0)
        step = b / torch.frexp(b)[0] / 4
        c = torch.round(q / step) * step
    else:
        c = torch.round(q)
    return (c.clamp(-top, top) * s).flatten(-2)


def _exact_entry_values(case, raw):
    """float64 K and V [T, H, D] of raw entries [T, entry_bytes], byte by byte."""
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
    e = raw[:, :h * unit].reshape(-1, h, unit).long()
    out = []
    for first, sfirst, g in ((0, d, case["k_scale"]), (d // 2, d + d // 16, case["v_scale"])):
        val = pairs[e[:, :, first:first + d // 2]].reshape(-1, h, d)
        out.append(val * scale[e[:, :, sfirst:sfirst + d // 16]].repeat_interleave(16, -1) * g)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_rope":
        table = s["cos_sin"].double().index_select(0, s["positions"].long())
        ang = torch.complex(table[:, :case["rotary"] // 2], table[:, case["rotary"] // 2:])[:, None, :]
        res = {}
        for name in ("q", "k"):
            x = s[name].double()
            if case["norm"]:
                x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / case["dim"] + 1e-6) * s[name + "_weight"].double()
            a, rest = x[..., :case["rotary"]], x[..., case["rotary"]:]
            if case["interleaved"]:
                w = torch.complex(a[..., 0::2].contiguous(), a[..., 1::2].contiguous()) * ang
                a = torch.view_as_real(w).flatten(-2)
            else:
                w = torch.complex(a[..., :case["rotary"] // 2].contiguous(), a[..., case["rotary"] // 2:].contiguous()) * ang
                a = torch.cat([w.real, w.imag], -1)
            res[name] = torch.cat([a, rest], -1)
        return res
    bs = case["block_size"]
    flat = s["pool"].reshape(-1, s["pool"].shape[-1])
    table = s["block_table"].long()
    if case["op"] == "kv_write":
        return {"k": _exact_values(case["kv"], s["k"].double() / case["k_scale"]) * case["k_scale"],
                "v": _exact_values(case["kv"], s["v"].double() / case["v_scale"]) * case["v_scale"]}
    if case["op"] == "kv_read":
        pos = s["token_pos"].long()
        k, v = _exact_entry_values(case, flat[table[s["token_batch"].long(), pos // bs] * bs + pos % bs])
        return {"k": k, "v": v}
    h, d, hq = case["heads_kv"], case["dim"], case["heads_q"]
    rows, n = s["indices"].shape
    out = torch.zeros((rows, hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((rows, hq), -math.inf, dtype=torch.float64, device="cuda")
    step = max(1, (1 << 26) // (n * h * d))
    for r0 in range(0, rows, step):
        idx = s["indices"][r0:r0 + step].long()
        m = idx.shape[0]
        at = idx.clamp(min=0)
        where = table[s["row_batch"][r0:r0 + step]].gather(1, at // bs) * bs + at % bs
        k, v = _exact_entry_values(case, flat[where.flatten()])
        k, v = (x.reshape(m, n, h, d).transpose(1, 2) for x in (k, v))  # [m, h, n, d]
        q = s["query"][r0:r0 + step].double().reshape(m, h, hq // h, d)
        z = torch.matmul(q, k.transpose(2, 3)) / math.sqrt(d)
        z = torch.where((idx >= 0)[:, None, None, :], z, torch.full_like(z, -math.inf))
        total = torch.logsumexp(z, -1, keepdim=True)
        w = torch.where(torch.isfinite(total), torch.exp(z - total), torch.zeros_like(z))
        out[r0:r0 + step] = torch.matmul(w, v).reshape(m, hq, d)
        lse[r0:r0 + step] = total.reshape(m, hq)
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}
