"""Forking in a hybrid model: the recurrent layers' states, a row each, go along with the pages of the attention layers."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_states_go_along(gpu_lib, dtype):
    glr, n, width, page, pages, cols = gpu_lib, 5, 128, 8, 12, 6
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    # rows 0 and 1 hold prompts of 11 and 16 tokens, row 4 one of 3
    lens = i32(11, 16, 0, 0, 3)
    table, shares = torch.zeros(n, cols, dtype=torch.int32, device="cuda"), torch.zeros(pages, dtype=torch.int32, device="cuda")
    free, count = i32(*range(pages)), i32(pages)
    cu = i32(0, 11, 27, 27, 27, 30)
    _, _, _, held, count, _ = glr.rglru_page_plan(0 * lens, cu, table, free, count, n_tokens=30, page_size=page)
    lam = rand(width)
    scan = lambda x, gx, ga, cu, h0: glr.rglru_fwd_varlen(x.to(dtype), gx.to(dtype), ga.to(dtype), lam, cu, None, h0, training=False)  # noqa: E731
    _, state, _ = scan(rand(30, width), rand(30, width), rand(30, width), cu, torch.zeros(n, width, device="cuda"))
    other = rand(n, 2, 16, 16)   # a state of another kind, for every row
    before = state.clone(), other.clone()
    # rows 2 and 3 go on from 1 and 0; row 4 holds tokens, so it is not served and stays as it is
    src = i32(-1, -1, 1, 0, 0)
    pairs, lens_out, held, count, unserved = glr.rglru_page_fork(src, lens, table, shares, free, count, page_size=page, held_lens=held)
    assert lens_out.tolist() == [11, 16, 16, 11, 3] and int(unserved) == 1
    rows = torch.stack([src, torch.arange(n, dtype=torch.int32, device="cuda")], 1)
    rows = torch.where((lens_out > lens)[:, None], rows, -1)
    glr.rglru_page_copy(rows, [state, other])
    for now, old in zip((state, other), before):
        assert torch.equal(now, old[[0, 1, 1, 0, 4]])
    # the next token, the same for all rows: a forked row goes on as its source does
    x, gx, ga = (rand(1, width).expand(n, width).contiguous() for _ in range(3))
    h, last, _ = scan(x, gx, ga, i32(0, 1, 2, 3, 4, 5), state)
    assert torch.equal(h[2], h[1]) and torch.equal(h[3], h[0]) and torch.equal(last[2], last[1]) and not torch.equal(h[4], h[0])
