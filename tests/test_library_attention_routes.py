"""Which sparse-attention calls go to the kernel of blocks of rows, and how they are laid out there: the host's
rule (no GPU needed), and that the calls of the GPU tests of that kernel do reach it on the GPU at hand."""
import ctypes

import pytest

import test_gpu_attention_rows as rows_tests

SMS = 152


@pytest.fixture(scope="module")
def route():
    from sparse_attention_token_block_gb300 import build as B
    B.build()
    import sparse_attention_token_block_gb300 as Q
    f = ctypes.CDLL(Q.TESTING_LIB_PATH).qli_testing_attention_rows

    def call(rows, hq, hkv, positions, k, batch=1, dim=128, with_k=True, sms=SMS, held=None, **kw):
        """None, or (rows of a block, KV heads of a CTA, positions of a mask)."""
        pages = -(-(held or positions) // 16)
        p = Q.make_problem(batch=batch, layout_q=Q.TND, total_q_tokens=rows, num_blocks=pages * batch, block_size=16,
                           max_blocks_per_seq=pages, sparse_count=k, sparse_mode=0, cmp_ratio=1, max_seqlen_q=rows,
                           max_seqlen_k=positions, **kw)
        a = Q.make_attention(num_heads_q=hq, num_heads_kv=hkv, head_dim=dim)
        shape = (ctypes.c_int32 * 3)()
        got = f(ctypes.byref(p), ctypes.byref(a), int(with_k), sms, shape)
        assert got in (0, 1), got
        return tuple(shape) if got else None
    return call


def test_the_rule(route):
    """Heads of 128, lists of 512 and a quarter of the positions, four blocks of rows a sequence, a block for
    every SM."""
    good = dict(rows=304, hq=64, hkv=8, positions=2048, k=512)
    assert route(**good) == (16, 1, 2048)
    for other in (dict(dim=64), dict(rows=288), dict(k=511, positions=2044), dict(positions=2049), dict(batch=5),
                  dict(hq=129, hkv=1), dict(sms=153)):
        assert route(**dict(good, **other)) is None, other
    # without lengths the table bounds the positions
    assert route(**dict(good, held=4096)) == (16, 1, 2048)
    assert route(**dict(good, held=4096, with_k=False)) is None
    assert route(**dict(good, held=4096, with_k=False, k=1024)) == (16, 1, 4096)


@pytest.mark.parametrize("hq,hkv,block,tiles", [(64, 8, 16, 64), (32, 8, 32, 48), (40, 8, 25, 61), (8, 8, 32, 48),
                                                (128, 1, 1, 64), (48, 8, 21, 64)])
def test_layouts(route, hq, hkv, block, tiles):
    """Rows of a block and tiles of 64 positions of a mask by the size of the group; heads of a CTA by the waves."""
    got = route(rows=SMS * block, hq=hq, hkv=hkv, positions=8000, k=2000)
    assert got == (block, max(1, hkv // 4), 64 * tiles)
    assert route(rows=8 * SMS * block, hq=hq, hkv=hkv, positions=8000, k=2000)[1] == hkv


def _of_the_gpu_tests(route, sms):
    """The layouts of the calls that the tests of this kernel make, for as many SMs."""
    mark = [m for m in rows_tests.test_head_layouts.pytestmark if m.args[0].startswith("hq")][0]
    for hq, hkv, q_lens in mark.args[1]:
        yield route(sum(q_lens), hq, hkv, 257, 512, len(q_lens), sms=sms), 1
    for k, keys in ((512, 4), (512, 129), (512, 64), (512, 2000), (2048, 2300)):
        yield route(330, 32, 16, keys, k, sms=sms), 1
    yield route(554, 64, 8, 201, 512, 4, sms=sms), 1
    for n, keys, k in ((320, 400, 512), (320, 190, 512), (304, 700, 700), (304, 200, 512), (304, 600, 512), (304, 2048, 512),
                       (304, 300, 512), (304, 256, 512)):
        yield route(n, 64, 8, keys, k, sms=sms), 1
    for n in (320, 310):
        yield route(n, 64, 8, 100, 512, 2, sms=sms), 1
    # several heads of a CTA
    for hq in (64, 32):
        for keys, k in ((5000, 1300), (900, 512)):
            yield route(sms * 1024 // hq, hq, 8, keys, k, 2, sms=sms), 2
    # repeats
    for keys, k in ((2300, 2048), (5000, 1300)):
        yield route(16 * -(-sms // 8), 64, 8, keys, k, sms=sms), 1
    yield route(16 * sms, 64, 8, 2300, 2048, sms=sms), 2
    # queries
    yield route(16 * -(-sms // 8), 64, 8, 600, 512, sms=sms), 1


def test_the_gpu_tests_reach_it(route):
    for i, (got, heads) in enumerate(_of_the_gpu_tests(route, SMS)):
        assert got is not None and got[1] == heads, (i, got)


@pytest.mark.gpu
def test_the_gpu_tests_reach_it_on_this_gpu(route):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    for i, (got, heads) in enumerate(_of_the_gpu_tests(route, torch.cuda.get_device_properties(0).multi_processor_count)):
        assert got is not None and got[1] == heads, (i, got)
