"""CPU checks of what the binding of the attention-step operators refuses: a tensor
that the kernels would read past its end or as another type."""
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def kq():
    import __graft_entry__

    __graft_entry__.build()
    import quantized_weight_streaming_gb300 as kq

    return kq


def test_qk_norm_refuses_tensors_that_its_kernels_would_misread(kq):
    w, rope = torch.ones(128), torch.zeros(50, 64)
    kq.QKNorm(4, 2, 128, 64, w, w, rope)
    kq.QKNorm(4, 2, 128, 64, None, None, rope)
    kq.QKNorm(4, 2, 128, 0, w, None, rope)  # without rotation the table is not looked at
    for bad in (w[:64], w.half(), w.double(), w.bfloat16(), torch.ones(256)[::2], torch.ones(128, 2), torch.ones(())):
        with pytest.raises(kq.KQError):
            kq.QKNorm(4, 2, 128, 64, bad, w, rope)
        with pytest.raises(kq.KQError):
            kq.QKNorm(4, 2, 128, 64, w, bad, rope)
    # a table of another width, type or layout: its rows end before what a position reads
    for bad in (torch.zeros(50, 32), rope.half(), rope.double(), torch.zeros(64, 50).T, torch.zeros(50, 128)[:, :64],
                torch.zeros(50 * 64)):
        with pytest.raises(kq.KQError):
            kq.QKNorm(4, 2, 128, 64, w, w, bad)
