"""Dense decode, eviction and their classes at the edges of what the calls
accept: alignment, ranges of weights and queries, tables that mix a sequence's
own pages with others, several streams.  References and bounds: dense_ref.py,
and the ones stated beside each test."""
import pytest
import torch

pytestmark = pytest.mark.gpu

qsa = pytest.importorskip("sparse_attention_decode_03_b200")

from tests.test_gpu_dense import Group, bits, i32, queries  # noqa: E402


@pytest.fixture(autouse=True, scope="module")
def _need_cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


# ---------------------------------------------------------------- alignment of the outputs


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hq,hkv", [(3, 1), (12, 1), (32, 2)])
def test_dense_decode_writes_outputs_that_are_8_byte_aligned(hq, hkv, fp8):
    """out and lse as slices of packed buffers: pairs of one tile, of several, and of several CTAs."""
    lens = [1, 3, 15, 16, 17, 40, 100, 9000, 2]
    grp = Group(lens, hkv, fp8, seed=hq)
    nq, n = len(lens), len(lens) * hq * 256
    q, q_seq, q_pos = queries(nq, hq, 1).cuda(), i32(list(range(nq))), i32([x - 1 for x in lens])
    ws = torch.empty(qsa.dense_decode_workspace_bytes(grp.cache, nq, hq), dtype=torch.uint8, device="cuda")
    got = []
    for shift in (0, 4):                              # elements: 0 and 8 bytes past a 256-byte boundary
        buf = torch.full((n + 8,), 7.0, dtype=torch.bfloat16, device="cuda")
        stats = torch.full((nq * hq + 2,), 7.0, device="cuda")
        out, lse = buf[shift:shift + n].view(nq, hq, 256), stats[shift // 4:shift // 4 + nq * hq].view(nq, hq)
        assert out.data_ptr() % 16 == 2 * shift
        qsa.qsa_dense_decode(grp.cache, q, q_seq, q_pos, 1 / 16, out, lse, ws)
        torch.cuda.synchronize()
        got.append((bits(out), bits(lse)))
        assert (buf[:shift] == 7.0).all() and (buf[shift + n:] == 7.0).all()       # nothing beside the rows
        assert (stats[:shift // 4] == 7.0).all() and (stats[shift // 4 + nq * hq:] == 7.0).all()
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
