"""Sizes at the end of what a launch holds, and arguments that are no matrices: refused before anything would be enqueued."""
import pytest
import torch

fc = pytest.importorskip("long_fft_convolution_amd")

UNSUPPORTED = 2


@pytest.mark.parametrize("N", [(1 << 28) - 15, (1 << 28) - 8, (1 << 28) - 1])
def test_columns_that_fill_a_launch_are_refused(N):
    # 16 columns a workgroup of 256 threads: 2^28 - 15 columns and more are 2^24 workgroups, 2^32 threads
    lib = fc.lib()
    a = 0x10000000000
    assert lib.fftconv_linear_fwd(a, 2 * a, None, None, 3 * a, None, None, 1, N, 1, 0, 2, None, 0, None) == UNSUPPORTED
    assert "too large" in fc.fftconv_last_error()
    assert lib.fftconv_linear_bwd(a, 2 * a, 3 * a, None, None, None, 4 * a, None, 8, N, 1, 0, 2, 5 * a, 1 << 39, None) == UNSUPPORTED
    assert "too large" in fc.fftconv_last_error()


@pytest.mark.gpu
def test_most_columns_of_a_launch():
    N = (1 << 28) - 16
    print(f"[case] one row, {N} columns", flush=True)
    W = torch.arange(256, dtype=torch.float32, device="cuda").to(torch.bfloat16).repeat(N // 256 + 1)[:N].view(N, 1)
    out = fc.linear_act(torch.full((1, 1), 2.0, dtype=torch.bfloat16, device="cuda"), W)
    assert torch.equal(out[0], (2.0 * W[:, 0].float()).to(torch.bfloat16))
