"""kvc_i4_attn over positions at the ends of int32, against the 64-bit definition."""
import pytest
import torch

from test_gpu_i4_cache import Cache, check_attention, i32, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from budgeted_kv_cache_gb300 import build
    build.build()
    import budgeted_kv_cache_gb300 as lib
    lib.library()
    return lib


@pytest.mark.parametrize("window", [0, 2 ** 31 - 1])
@pytest.mark.parametrize("d, n_q", [(128, 1), (64, 5)])
def test_distances_past_31_bits(kvc, d, n_q, window):
    """A query at the largest position, keys over the whole range of int32: distances of up to 2^32 - 1."""
    c = Cache(kvc, 1, 1, 2, d, 200, [200], 0, 3, 8)
    far = torch.randint(-2 ** 31, 2 ** 31, c.rows.pos.shape, generator=c.g, device="cuda")
    far[:, :50] = -2 ** 31 + torch.arange(50, device="cuda")
    c.rows.pos.copy_(far)
    slopes = torch.rand(8, generator=c.g, device="cuda") * 1e-9                # biases of up to 4.3
    q_pos = i32([[2 ** 31 - 1 - i for i in range(n_q)]])
    q = randn(c.g, 1, 1, 8, n_q, d)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:-1], device="cuda")
    ws = torch.empty(max(1, kvc.kvc_i4_attn_workspace_bytes(c.shape, c.rows, n_q, True)), dtype=torch.uint8, device="cuda")
    mass0 = c.rows.mass.clone()
    kvc.kvc_i4_attn(c.shape, c.rows, q, out, q_pos=q_pos, mods=kvc.ScoreMods(0.0, slopes, window), add_mass=True,
                    row_lse=lse, workspace=ws)
    check_attention(c, q, out, lse, mass0, q_pos, 0.0, slopes, window, None, True)
