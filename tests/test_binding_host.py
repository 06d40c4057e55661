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


class Second(torch.Tensor):
    """A tensor in host memory that says it lies on the second GPU."""
    device = property(lambda self: torch.device("cuda", 1))


class FakeStream:
    def __init__(self, index):
        self.device, self.cuda_stream = torch.device("cuda", index), 70 + index


@pytest.fixture
def two_gpus(ssm, monkeypatch):
    """The first GPU is current, every tensor lies on the second; C entry points that launch only note how they were
    called: (name, the current device, the stream's address)."""
    now, noted, real = [0], [], ssm.lib()

    class On:
        def __init__(self, device):
            self.index = torch.device(device).index

        def __enter__(self):
            self.before, now[0] = now[0], self.index

        def __exit__(self, *_):
            now[0] = self.before

    def note(name):
        def f(*args):
            s = args[-1]
            noted.append((name, now[0], s.value if hasattr(s, "value") else s))
            return 0
        return f

    class Library:
        def __getattr__(self, name):
            return getattr(real, name) if name.endswith(("_bytes", "_elems")) else note(name)

        __getitem__ = __getattr__

    for name in ("empty", "zeros", "full"):
        make = getattr(torch, name)
        monkeypatch.setattr(torch, name, lambda *a, _make=make, device=None, **k: _make(*a, **k).as_subclass(Second))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", On)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: On(s.device))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d: FakeStream(torch.device(d).index))
    monkeypatch.setattr(ssm, "_current_raw_stream", lambda index: 70 + index)
    monkeypatch.setattr(ssm, "lib", lambda: Library())
    monkeypatch.setattr(ssm, "_short", False)
    for e in vars(ssm).values():
        if isinstance(e, ssm._Entry):
            monkeypatch.setattr(e, "f", note(e.name))
    return noted


def every_call(ssm):
    """All calls that launch, by the name of their C entry point: each takes the stream."""
    def new(*shape, dtype=torch.float32):
        return torch.ones(*shape, dtype=dtype).as_subclass(Second)
    bf, ws = torch.bfloat16, ssm.Workspace.of_bytes(1 << 20, "cuda:1")
    x, A, Bm, r = new(2, 16, 16), new(16, 16), new(2, 16, 16), new(2, 16)
    cell, gate, st = new(1, 1, 64, 128, dtype=bf), new(1, 1, 64, 128), new(1, 1, 128, 128)
    one, g1, m = new(1, 1, 128, dtype=bf), new(1, 1, 128), (st, new(1, 1, 128), new(1, 1))
    a, w, ids, lam = new(4, 16, dtype=bf), new(8, 16, dtype=bf), new(2, dtype=torch.int64), new(16)
    q, sc, ck = new(8, 16, dtype=torch.uint8), new(8, 1, dtype=bf), new(1 << 14)
    return {
        "ssm_scan_fwd": lambda s: ssm.scan_fwd(x, x, A, Bm, Bm, stream=s),
        "ssm_scan_bwd": lambda s: ssm.scan_bwd(x, x, A, Bm, Bm, x, ck, stream=s),
        "ssm_step": lambda s: ssm.step(new(2, 16, 16), r, r, A, r, r, stream=s),
        "ssm_dA_log_grad": lambda s: ssm.dA_log_grad(A, A, stream=s),
        "ssm_conv1d_fwd": lambda s: ssm.conv1d_fwd(x, new(16, 4), stream=s),
        "ssm_conv1d_bwd": lambda s: ssm.conv1d_bwd(x, new(16, 4), x, stream=s),
        "ssm_dtproj_fwd": lambda s: ssm.dtproj_fwd(a, w, stream=s),
        "ssm_dtproj_bwd": lambda s: ssm.dtproj_bwd(a, w, new(4, 8), stream=s),
        "gdn2_chunk_fwd": lambda s: ssm.gdn2_fwd(cell, cell, cell, gate, cell, cell, stream=s),
        "gdn2_step": lambda s: ssm.gdn2_step(one, one, one, g1, one, one, st, stream=s),
        "mlstm_chunk_fwd": lambda s: ssm.mlstm_fwd(cell, cell, cell, new(1, 1, 64), new(1, 1, 64), stream=s),
        "mlstm_step": lambda s: ssm.mlstm_step(one, one, one, new(1, 1), new(1, 1), m, stream=s),
        "ssm_glr_fwd": lambda s: ssm.glr_fwd(x, x, x, lam, stream=s),
        "ssm_glr_bwd": lambda s: ssm.glr_bwd(x, x, x, lam, x, ck, stream=s),
        "ssm_glr_step": lambda s: ssm.glr_step(new(2, 16), r, r, r, lam, stream=s),
        "ssm_layernorm_fwd": lambda s: ssm.layer_norm_fwd(r, lam, stream=s),
        "ssm_layernorm_bwd": lambda s: ssm.layer_norm_bwd(r, r, new(2), new(2), lam, stream=s),
        "ssm_embed_fwd": lambda s: ssm.embed_fwd(ids, A, stream=s),
        "ssm_embed_bwd": lambda s: ssm.embed_bwd(ids, r, 8, stream=s),
        "ssm_w4_quantize": lambda s: ssm.w4_quantize(new(8, 32), 32, stream=s),
        "ssm_w4_matvec": lambda s: ssm.w4_matvec(new(2, 32, dtype=bf), q, sc, stream=s),
        "ssm_exp2_fma": lambda s: ssm.exp2_fma(r, stream=s),
        "ssm_poll_status": lambda s: ssm.poll_status(ws, stream=s),
        "ssm_clear_status": lambda s: ssm.clear_status(ws, stream=s),
    }


def test_calls_are_made_on_their_tensors_device(ssm, two_gpus):
    for name, call in every_call(ssm).items():
        for stream in (None, FakeStream(1)):
            two_gpus.clear()
            call(stream)
            assert two_gpus == [(name, 1, 71)], name


def test_a_stream_of_another_device_is_refused(ssm, two_gpus):
    for name, call in every_call(ssm).items():
        two_gpus.clear()
        with pytest.raises(ValueError, match="stream is on cuda:0"):
            call(FakeStream(0))
        assert not two_gpus, name


def test_no_cuda_device(ssm):
    with pytest.raises(ValueError, match="CUDA"):
        ssm.poll_status(ssm.Workspace.of_bytes(256, "cpu"))


@pytest.mark.parametrize("built_for", [None, "torch 1.0.0 True cpython-312-x86_64-linux-gnu", "2.0.1"])
def test_a_short_way_built_for_another_torch_is_not_loaded(ssm, monkeypatch, tmp_path, built_for):
    from selective_state_space_07_gb300 import _builder
    note = tmp_path / "built_for.txt"
    if built_for is not None:
        note.write_text(built_for)
    monkeypatch.setattr(_builder, "BINDING_TORCH", str(note))
    monkeypatch.setattr(ssm, "_short", None)
    assert not ssm._short_way() and _builder.binding_stale()


def test_the_short_way_that_build_made_is_loaded(ssm, monkeypatch):
    from selective_state_space_07_gb300 import _builder
    if not _builder.binding_fits():
        pytest.skip("the short way was not built here")
    monkeypatch.setattr(ssm, "_short", None)
    assert ssm._short_way() is ssm._binding and not _builder.binding_stale()
