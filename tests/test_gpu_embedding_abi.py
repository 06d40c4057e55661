"""The embedding gradient through its C boundary, where Python's checks do not
stand before it."""
import ctypes

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ssm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import selective_state_space_07_gb300 as m
    m.build()
    return m


@pytest.mark.parametrize("tokens", [40, 40000])  # sorted straight, and divided among the ranges first
@pytest.mark.parametrize("padding,zero", [(5, 5), (-1, None), (-(1 << 40), None), (9, None), ((1 << 32) + 5, None), ((1 << 40) + 5, None)])
def test_a_padding_id_outside_the_table_is_none(ssm, padding, zero, tokens):
    V, D = 9, 8
    ids, dy = torch.arange(tokens, device="cuda") % V, torch.ones(tokens, D, device="cuda")
    dW = torch.full((V, D), -1.0, device="cuda")
    n = ssm.embed_workspace_bytes(tokens, V, D)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    a = ssm.EmbedBwdArgs(tokens=tokens, V=V, D=D, padding_id=padding, io_dtype=0, ids64=1, scale=1.0, pad_=0, ids=ids.data_ptr(),
                         dy=dy.data_ptr(), dW=dW.data_ptr(), workspace=ws.data_ptr(), workspace_bytes=n, status=None)
    assert ssm.lib().ssm_embed_bwd(ctypes.byref(a), torch.cuda.current_stream().cuda_stream) == 0
    want = torch.bincount(ids, minlength=V).float()
    if zero is not None:
        want[zero] = 0
    assert torch.equal(dW, want[:, None].expand(V, D))
