"""The list operators at the edges of what their calls allow."""
import ctypes

import pytest
import torch

import precision_adam_optimizer_amd as pk
from tests.test_gpu_list import U

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("amp", [False, True])
@pytest.mark.parametrize("eps", [2.0 ** -149, 1e-42, 2.0 ** -139, 2.0 ** -138, 2.0 ** -126, 1e-35, 1e-30])
def test_tiny_eps(bits, amp, eps):
    """An eps that is subnormal in fp32, or near it: weights whose gradient was never anything but zero stay
    as they are, the others move by the formula (12u of the update, and the sum)."""
    gr = torch.tensor([0.0, -0.0, 1e-3, -1e-10, 1e-20, 0.0] + [0.0] * 1100, device="cuda")
    p = torch.ones(gr.numel(), device="cuda")
    opt = pk.AdamW([p], [gr], state_bits=bits)
    hp = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=eps, weight_decay=0.0)
    if amp:
        opt.step_amp(pk.amp_state(1.0), **hp)
    else:
        opt.step(step=1, **hp)
    zero = gr == 0
    assert bool((p[zero] == 1).all()), p[zero][:4]
    g = gr[~zero].double().cpu()
    v = (g * g).float().double()  # times 0.05, rounded, over 0.05: within 3u, and a step where it is subnormal
    upd = 1e-3 * g / (v.sqrt() + eps)
    some = v > 2.0 ** -120
    err = (p[~zero].double().cpu() - (1 - upd)).abs()
    assert bool((err <= U * (13 * upd.abs() + 1.01))[some].all()), err / U
    opt.close()


def test_an_old_error_of_the_runtime_is_not_a_launch_s():
    """The thread's last HIP error, from a call of the program's own, does not stop a step."""
    pk.load()
    with open("/proc/self/maps") as f:  # the runtime that this process has loaded
        hip = ctypes.CDLL(next(line.split()[-1] for line in f if "libamdhip64" in line))
    xs = [torch.ones(300, device="cuda") for _ in range(2)]
    gs = [torch.ones(300, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    opt = pk.AdamW(xs, gs, state_bits=[32, 8])
    amp = pk.amp_state(1.0)
    clip = pk.GradClip(gs, outs=[None, None])
    torch.cuda.synchronize()
    try:
        assert hip.hipSetDevice(10 ** 6) != 0  # no such device
        opt.step(lr=0.25, step=1)
        opt.step_amp(amp, lr=0.25)
        clip.clip(1.0)
    finally:
        hip.hipGetLastError()
    torch.cuda.synchronize()
    # 1 - 0.25 after the first step; the second takes 1.9 / sqrt(2) of its rate (less what 8 bits lose)
    assert all(bool((x == x[0]).all()) and 0.3 < float(x[0]) < 0.5 for x in xs), [x[0] for x in xs]
    assert pk.read_amp_state(amp)["step"] == 1
    opt.close()
    clip.close()
