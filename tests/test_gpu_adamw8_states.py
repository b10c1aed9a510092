"""The states of AdamW in 8 bits against their formula, code for code."""
import pytest
from test_gpu_block import random_bits, state_values
from test_gpu_layer import gen_for, normal, ops, torch  # noqa: F401 (fixtures)
pytestmark = pytest.mark.gpu


# the largest gradient's power of ten and from one block of 32 to the next; 1e-15 squared lies below 2^-64, where the root moves numbers up
@pytest.mark.parametrize("dtype,top,apart", [("bfloat16", 0, 1), ("float16", 3, 1), ("float32", 0, 1), ("bfloat16", 3, 3), ("float32", 3, 3)])
def test_adamw8_states_follow_the_formula_bit_for_bit(torch, ops, dtype, top, apart):
    """Whatever the parameters' type: every operation of the moments rounded to fp32 as torch's are, in millions of elements."""
    gen = gen_for(torch, 23)
    n = 3_000_000
    dt = getattr(torch, dtype)
    p = normal(torch, gen, n).to(dt)
    state = ops.adamw8_state(p)
    scale = 10.0 ** (apart * (torch.arange(n, device="cuda") // 32 % 7 - 6) + top)
    for step in (1, 2, 3):
        g = (normal(torch, gen, n) * scale).clamp(-6e4, 6e4).to(dt)
        held = [state_values(torch, state[i], state[i + 1]).float() for i in (0, 2)]
        ops.adamw8_step([p], [g], [state], lr=1e-3, step=step, beta1=0.9, beta2=0.95, seed=78)
        f = g.float()
        m = 0.9 * held[0] + (1 - 0.9) * f
        r = torch.sqrt(0.95 * held[1].square() + (1 - 0.95) * (f * f))
        for val, i, rnd, least in zip((m, r), (0, 2), random_bits(torch, 78, step, 0, n), (0.0, 2.0 ** -9)):
            byte = state[i + 1].view(torch.uint8).repeat_interleave(32)[:n]
            x = (val.abs().double() * torch.exp2(127 - byte.double())).float()
            fine = torch.floor(x.double() * 512 + rnd.double() * 2.0 ** -16) * 2.0 ** -9
            size = torch.where(x < 2.0 ** -6, fine.float(), ((x.view(torch.int32) + (rnd.int() << 4)) & ~0xfffff).view(torch.float32))
            size = torch.where((val != 0) & (size < least), torch.full_like(size, least), size)
            off = state[i].view(torch.float8_e4m3fn).float().abs() != size
            # below 2^-6 the number is added to 2^-6 first, one rounding more of 2^-31: a code in 2^16 of them may end elsewhere, and fewer do
            assert not (off & (x >= 2.0 ** -6)).any() and off.sum() <= 1 + 1e-5 * (x < 2.0 ** -6).sum(), (step, i, int(off.sum()))
