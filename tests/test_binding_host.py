"""What the Python binding refuses before it calls the library: host tensors,
and work for another GPU than the one that launches go to."""

import pytest
import torch

from integer_only_dnn_amd import ie


def test_streams_are_those_of_the_current_gpu(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 1000 + index, raising=False)
    assert ie._stream(torch.device("cuda")) == 1000 and ie._stream(torch.device("cuda:0")) == 1000
    with pytest.raises(ValueError):
        ie._stream(torch.device("cpu"))
    with pytest.raises(ValueError):
        ie._stream(torch.device("cpu:0"))
    for _ in range(2):
        with pytest.raises(ValueError):
            ie._stream(torch.device("cuda:1"))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    assert ie._stream(torch.device("cuda")) == 1001 and ie._stream(torch.device("cuda:1")) == 1001


def test_host_matrices_are_refused():
    m = ie.Mat.empty(4, 8, ie.ROW, device="cpu")
    with pytest.raises(ValueError):
        m.c()
    with pytest.raises(ValueError):
        m.c(2, 16)
    with pytest.raises(ValueError):
        ie.ie_relu_fwd(m, m)


def test_workspace_follows_its_buffer():
    """A buffer that the caller puts in, or takes away, is the one that calls get."""
    ws = ie.Workspace("cpu")
    for n in (512, 1024):
        ws.buf = torch.zeros(n, dtype=torch.uint8)
        assert ws.get(300) == (ws.buf.data_ptr(), n)
    ws.buf = None
    assert ws.status() == 0
    with pytest.raises(ValueError):  # asked for anew, and refused: host memory
        ws.get(700)
    assert ws.buf.numel() == 700


@pytest.mark.parametrize("eps", [(128, 0), (-129, 0), (85, -140), (85, 128), (85,), (1, 2, 3)])
def test_eps_that_is_no_scalar_is_refused(eps):
    """A byte would wrap: 85 * 2^-140 would be read as 85 * 2^116."""
    with pytest.raises(ValueError):
        ie.ie_layer_norm_fwd(None, None, None, eps, None, None)
    with pytest.raises(ValueError):
        ie.ie_layer_norm_bwd(None, None, None, eps, None, None, None, None)


class _OnGpu(torch.Tensor):
    """A host tensor that says it is on the GPU: descriptors only take its address."""
    is_cuda = property(lambda self: True)


def _gpu(*shape):
    return torch.zeros(shape, dtype=torch.int8).as_subclass(_OnGpu)


def test_descriptors_hold_their_matrix():
    """Fewer exponents than groups, or fewer mantissas than the view, would be read past their end."""
    for rows, cols, n, group, ok in ((4, 8, 4, ie.ROW, True), (4, 8, 1, ie.ROW, False), (4, 8, 3, ie.ROW, False),
                                     (4, 8, 1, ie.TENSOR, True), (4, 8, 0, ie.TENSOR, False), (8, 1, 1, ie.ROW, False),
                                     (1, 8, 1, ie.ROW, True), (0, 8, 0, ie.ROW, True), (0, 8, 0, ie.TENSOR, False)):
        m = ie.Mat(_gpu(rows, cols), _gpu(n), group)
        if ok:
            d = m.c()
            assert (d.rows, d.cols, d.group) == (rows, cols, group)
        else:
            with pytest.raises(ValueError):
                m.c()
    image = ie.Mat(_gpu(2, 3, 3, 16), _gpu(1), ie.TENSOR)
    assert image.c(18, 16).rows == 18
    for view in ((18, 17), (19, 16)):
        with pytest.raises(ValueError):
            image.c(*view)
    with pytest.raises(ValueError):
        ie.Mat(_gpu(2, 3, 3, 16), _gpu(2), ie.ROW).c(18, 16)
