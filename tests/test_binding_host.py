"""What the Python binding of the language-model operators refuses or decides
on the host, without a GPU."""
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ssm():
    import selective_state_space_07_gb300 as m
    m.build()
    return m


def test_a_status_word_lies_on_the_calls_device(ssm):
    ws = ssm.Workspace.of_bytes(256, "cpu")
    assert ssm._status(None, torch.device("cuda", 0)) == 0
    assert ssm._status(ws, torch.device("cpu")) == ws.buf.data_ptr()
    with pytest.raises(ValueError, match="workspace is on cpu"):
        ssm._status(ws, torch.device("cuda", 0))


def test_a_scans_workspace_lies_on_the_calls_device(ssm):
    ws = ssm.Workspace(1, 8, 8, "cpu")
    assert ssm._ws(ws, 1, 8, 8, torch.device("cpu")) is ws
    with pytest.raises(ValueError, match="workspace is on cpu"):
        ssm._ws(ws, 1, 8, 8, torch.device("cuda", 0))
