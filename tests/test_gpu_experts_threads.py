"""Two host threads that call the operators for experts of another form at the same time, each on its own
stream, get the bits that one thread gets: the checks of a signature, the kernels' attributes and the
workspaces are nobody's state that two calls could meet in."""
import threading

import pytest
import torch

from moe_ffn_expert_gb300 import expert_ops, grad_ops

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def case(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T, K, E, H, I = 300 + seed, 2, 6 + seed, 136, 264
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)
    ids = torch.randint(-1, E, (T, K), generator=g, device="cuda")
    return ids, E, randn(T, H), randn(E, H, I), randn(E, I, H), torch.rand(T, K, generator=g, device="cuda")


def step(ids, E, x, w1, w2, weights):
    table = expert_ops.expert_table(ids, E)
    rows = expert_ops.dispatch_forward(x, table)
    h = expert_ops.grouped_mm_forward(rows, w1, table.offsets)
    o = expert_ops.grouped_mm_forward(h, w2, table.offsets)
    y = expert_ops.combine_forward(o, table, weights)
    do, dw = expert_ops.combine_backward(y, o, table, weights)
    dh, dw2 = expert_ops.grouped_mm_backward(do, h, w2, table.offsets, weight_grad_dtype=torch.float32)
    dr, dw1 = expert_ops.grouped_mm_backward(dh, rows, w1, table.offsets)
    grads = [dw1, dw2, expert_ops.combine_forward(dr, table)]
    norm = grad_ops.clip_grad_norm(grads, 1.0)
    return (*table[:3], y, dw, norm, *grads)


def test_two_threads_at_once():
    cases = [case(seed) for seed in range(2)]
    want = [step(*c) for c in cases]
    torch.cuda.synchronize()
    errors, wrong = [], [0, 0]

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for n in range(30):
                    if n % 10 == 0:  # signatures that nobody knows any more
                        expert_ops._grouped_plans.clear()
                        expert_ops._row_plans.clear()
                    for got, ref in zip(step(*cases[i]), want[i]):
                        wrong[i] += int((got != ref).sum())
        except Exception as error:  # told by the main thread
            errors.append(error)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors and wrong == [0, 0]
