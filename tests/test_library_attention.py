"""Refusals of the attention-side entry points and the layout of their attribute structs: everything
here is checked on the host before any CUDA call, so no GPU is needed."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
X = 1 << 20                                       # a 256-byte aligned stand-in address, never dereferenced


@pytest.fixture(scope="module")
def Q():
    from sparse_attention_token_block_gb300 import build as B
    B.build()
    import sparse_attention_token_block_gb300 as Q
    return Q


def _problem(Q, **kw):
    args = dict(batch=2, max_q_tokens=1, num_blocks=8, block_size=64, max_blocks_per_seq=4, sparse_count=64,
                sparse_mode=3, cmp_ratio=1, max_seqlen_q=1, max_seqlen_k=256)
    args.update(kw)
    return Q.make_problem(**args)


def _attention(Q, **kw):
    args = dict(num_heads_q=16, num_heads_kv=2, head_dim=128)
    args.update(kw)
    return Q.make_attention(**args)


def _rotation(Q, **kw):
    args = dict(num_heads_q=4, num_heads_k=1, head_dim=128, rotary_dim=64, max_positions=100)
    args.update(kw)
    return Q.make_norm_rope(**args)


def test_defaults_are_valid(Q):
    a, r = Q.Attention(), Q.Rotation()
    Q.lib.qli_attention_init(ctypes.byref(a))
    Q.lib.qli_rotation_init(ctypes.byref(r))
    assert Q.validate_attention(a)[0] == 0 and Q.validate_norm_rope(r)[0] == 0
    assert Q.kv_entry_bytes(a) == 8 * 144
    assert Q.kv_entry_bytes(_attention(Q, head_dim=64, num_heads_q=3, num_heads_kv=3)) == 224       # 3 * 72 up to 16
    Q.lib.qli_attention_init(None)
    Q.lib.qli_rotation_init(None)
    assert Q.lib.qli_attention_validate(None, None) == 1 and Q.lib.qli_rotation_validate(None, None) == 1
    assert Q.lib.qli_kv_entry_bytes(None) == 0


@pytest.mark.parametrize("field,value", [
    ("num_heads_kv", 0), ("num_heads_kv", 65), ("num_heads_q", 17), ("num_heads_q", 0), ("num_heads_q", 258),
    ("head_dim", 96), ("head_dim", 256), ("dtype", 2), ("kv_dtype", -1), ("softmax_scale", -1.0),
    ("softmax_scale", float("nan")), ("softmax_scale", float("inf")), ("k_scale", 0.0), ("k_scale", 1e-40),
    ("v_scale", -2.0), ("v_scale", float("nan")), ("k_scale", float("inf")), ("kv_stride", -16), ("kv_stride", 8)])
def test_attention_attributes_rejected(Q, field, value):
    a = _attention(Q)
    setattr(a, field, value)
    st, why = Q.validate_attention(a)
    assert st == 1 and why != "ok"
    assert Q.kv_entry_bytes(a) == 0
    p = _problem(Q)
    assert Q.lib.qli_sparse_attention(ctypes.byref(p), ctypes.byref(a), X, 0, None, X, X, X, X, X, None, None, 0, None) == 1
    assert Q.lib.qli_kv_write(ctypes.byref(p), ctypes.byref(a), 1, X, 0, X, 0, X, X, X, X, None, 0, None) == 1
    assert Q.lib.qli_kv_read(ctypes.byref(p), ctypes.byref(a), 1, X, X, X, X, X, 0, X, 0, None, 0, None) == 1


@pytest.mark.parametrize("field,value", [
    ("num_heads_q", -1), ("num_heads_q", 1025), ("num_heads_k", -1), ("num_heads_k", 1025), ("head_dim", 32),
    ("rotary_dim", 4), ("rotary_dim", 136), ("rotary_dim", -8), ("max_positions", 0), ("dtype", 2), ("interleaved", 2),
    ("norm", -1), ("eps", -1e-6), ("eps", float("nan")), ("eps", float("inf"))])
def test_rotation_attributes_rejected(Q, field, value):
    r = _rotation(Q)
    setattr(r, field, value)
    st, why = Q.validate_norm_rope(r)
    assert st == 1 and why != "ok"
    assert Q.lib.qli_norm_rope(ctypes.byref(r), 1, X, 0, X, 0, X, X, X, X, X, 0, X, 0, None, 0, None) == 1


def test_norm_rope_arguments_rejected(Q):
    r = _rotation(Q)
    names = ["tokens", "q", "qs", "k", "ks", "qw", "kw", "pos", "cs", "qo", "qos", "ko", "kos", "ws", "wsb", "st"]
    good = dict(tokens=3, q=X, qs=0, k=X, ks=0, qw=X, kw=X, pos=X, cs=X, qo=X, qos=0, ko=X, kos=0, ws=None, wsb=0, st=None)

    def call(rr=r, **kw):
        v = dict(good, **kw)
        return Q.lib.qli_norm_rope(ctypes.byref(rr), *[v[n] for n in names])
    for bad in (dict(tokens=-1), dict(tokens=(1 << 30) + 1), dict(q=None), dict(k=None), dict(qo=None), dict(ko=None),
                dict(qw=None), dict(kw=None), dict(pos=None), dict(pos=X + 2), dict(cs=None), dict(cs=X + 8),
                dict(q=X + 8), dict(k=X + 2), dict(qo=X + 8), dict(ko=X + 8), dict(qw=X + 2), dict(qs=504),
                dict(qs=516), dict(ks=120), dict(ks=-128), dict(qos=504), dict(kos=132), dict(ws=X, wsb=64),
                dict(ws=X + 16, wsb=256)):
        assert call(**bad) == 1, bad
    assert call(tokens=0, q=None, k=None, qo=None, ko=None, qw=None, kw=None, pos=None, cs=None) == 0
    none = _rotation(Q, num_heads_q=0, num_heads_k=0)
    assert call(none, q=None, k=None) == 0


def test_kv_arguments_rejected(Q):
    p, a = _problem(Q), _attention(Q)
    page = 64 * 288
    wn = ["n", "k", "ks", "v", "vs", "tb", "tp", "bt", "kv", "ws", "wsb", "st"]
    rn = ["n", "tb", "tp", "bt", "kv", "k", "ks", "v", "vs", "ws", "wsb", "st"]
    good = dict(n=3, k=X, ks=0, v=X, vs=0, tb=X, tp=X, bt=X, kv=X, ws=None, wsb=0, st=None)

    def both(pp=p, aa=a, **kw):
        v = dict(good, **kw)
        w = Q.lib.qli_kv_write(ctypes.byref(pp), ctypes.byref(aa), *[v[n] for n in wn])
        r = Q.lib.qli_kv_read(ctypes.byref(pp), ctypes.byref(aa), *[v[n] for n in rn])
        assert w == r
        return w
    for bad in (dict(n=-1), dict(n=(1 << 30) + 1), dict(k=None), dict(v=None), dict(tb=None), dict(tp=None),
                dict(bt=None), dict(kv=None), dict(k=X + 8), dict(v=X + 8), dict(kv=X + 8), dict(ks=248), dict(vs=260),
                dict(ws=X, wsb=128), dict(ws=X + 128, wsb=256)):
        assert both(**bad) == 1, bad
    assert both(n=0, k=None, v=None, tb=None, tp=None, bt=None, kv=None) == 0
    assert both(aa=_attention(Q, kv_stride=page - 16)) == 1
    bad = _problem(Q)
    bad.block_size = 24
    assert both(pp=bad) == 1


def test_sparse_attention_arguments_rejected(Q):
    names = ["q", "qs", "sq", "sk", "bt", "idx", "kv", "out", "lse", "ws", "wsb", "st"]
    good = dict(q=X, qs=0, sq=None, sk=X, bt=X, idx=X, kv=X, out=X, lse=X, ws=None, wsb=0, st=None)

    def call(p=None, a=None, **kw):
        v = dict(good, **kw)
        return Q.lib.qli_sparse_attention(ctypes.byref(p or _problem(Q)), ctypes.byref(a or _attention(Q)),
                                          *[v[n] for n in names])
    for bad in (dict(q=None), dict(idx=None), dict(out=None), dict(bt=None), dict(kv=None), dict(q=X + 8),
                dict(kv=X + 8), dict(out=X + 8), dict(lse=X + 2), dict(qs=2040), dict(qs=2052), dict(ws=X, wsb=16),
                dict(ws=X + 64, wsb=256)):
        assert call(**bad) == 1, bad
    assert call(a=_attention(Q, kv_stride=64 * 288 - 16)) == 1
    assert call(p=_problem(Q, layout_q=Q.TND, total_q_tokens=5)) == 1                  # no prefix sums
    assert call(p=_problem(Q, max_q_tokens=0), q=None, idx=None, out=None) == 0         # no rows
    assert call(p=_problem(Q, batch=2, max_q_tokens=1 << 24, max_seqlen_k=16)) == 2     # beyond the grid
    bad = _problem(Q)
    bad.sparse_count = 0
    assert call(p=bad) == 1


def test_binding_refuses_tensors_that_do_not_fit(Q):
    torch = pytest.importorskip("torch")
    r = _rotation(Q)
    pos = torch.zeros(3, dtype=torch.int32)
    q, k, w = torch.zeros(3, 4, 128, dtype=torch.bfloat16), torch.zeros(3, 1, 128, dtype=torch.bfloat16), torch.zeros(128)
    cs = torch.zeros(100, 64)

    def call(q=q, k=k, qo=q, ko=k):
        return Q.norm_rope(r, q, k, w, w, pos, cs, qo, ko, stream=0)
    with pytest.raises(TypeError):
        call(q=q.half())
    for bad in (q[:2], q[:, :3], q.transpose(1, 2).contiguous().transpose(1, 2), q[:1].expand(3, 4, 128)):
        with pytest.raises(ValueError):
            call(q=bad)
    p, a = _problem(Q, batch=3), _attention(Q, num_heads_q=4, num_heads_kv=1)
    idx = torch.zeros(3, 64, dtype=torch.int32)
    packed = torch.zeros(3, 6, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):                                                   # a strided output
        Q.sparse_attention(p, a, q, None, idx, idx, idx, idx, packed[:, :4], stream=0)
    with pytest.raises(ValueError):                                                   # rows
        Q.sparse_attention(p, a, q[:2], None, idx, idx, idx, idx, q, stream=0)


def test_struct_layouts_match_the_header(Q, tmp_path):
    for struct, cls in (("qli_rotation", Q.Rotation), ("qli_attention", Q.Attention)):
        fields = [f[0] for f in cls._fields_]
        src = tmp_path / (struct + ".c")
        src.write_text("#include <stddef.h>\n#include <stdio.h>\n#include \"qli.h\"\nint main(void) {\n"
                       "  printf(\"%%zu\\n\", sizeof(%s));\n" % struct
                       + "".join("  printf(\"%%zu\\n\", offsetof(%s, %s));\n" % (struct, f) for f in fields)
                       + "  return 0;\n}\n")
        exe = tmp_path / struct
        subprocess.check_call(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(src)])
        got = [int(x) for x in subprocess.check_output([str(exe)]).split()]
        assert got[0] == ctypes.sizeof(cls)
        assert got[1:] == [getattr(cls, f).offset for f in fields]
