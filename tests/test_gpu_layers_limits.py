"""GPU tests of the gated recurrence and the layer norm, and of the one-token
steps, at the ends of their sizes and of float32's range."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import selective_state_space_28_amd as ssm
    ssm.load()
    return torch.device("cuda:0")


def test_steps_of_the_largest_batch(dev):
    """2^31 - 1 sequences of one channel, in launches of 65535: tokens at both ends and in the middle are those of a
    call on them alone, in the gated and in the selective step."""
    import torch
    import selective_state_space_28_amd as ssm
    if torch.cuda.mem_get_info()[0] < 60 * 2**30:
        pytest.skip("needs 60 GiB of GPU memory")
    n = 2**31 - 1
    windows = [slice(at, at + 9) for at in (0, 2**30 + 1, 32767 * 65535 - 4, 32768 * 65535 - 4, n - 9)]
    gen = torch.Generator(device=dev)
    gen.manual_seed(9)
    x = torch.empty((n, 1), dtype=torch.bfloat16, device=dev)
    for k in range(0, n, 2**28):
        x[k:k + 2**28].normal_(generator=gen)
    A = torch.full((1,), -0.7, device=dev)

    def check(step, *tok):
        state = torch.ones((n, 1) + A.shape[1:], device=dev)
        y = step(state, *tok, torch.full_like(x, float("nan")))
        for s in windows:
            few = torch.ones((9, 1) + A.shape[1:], device=dev)
            want = step(few, *(v[s].contiguous() for v in tok), torch.empty_like(x[s]))
            assert torch.equal(y[s], want) and torch.equal(state[s], few), s
        for k in range(0, n, 2**28):
            assert not bool(y[k:k + 2**28].isnan().any()), k

    check(lambda st, u, out: ssm.ssm_gated_state_update(st, u, u, A, out=out), x)
    A = A.view(1, 1)
    check(lambda st, u, out: ssm.ssm_state_update(st, u, u, A, u, u, out=out), x)
