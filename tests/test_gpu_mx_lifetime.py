"""On the GPU: memory of an optimiser group that has gone is not handed out
while a step of it is still to run on another stream."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_tables_are_not_handed_out_before_the_step_on_another_stream():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from layer_streamed_qlora_b200 import _lib as L
    n, hp = 4096, dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, grad_scale=1.0, t=1)
    g = torch.from_numpy(np.random.default_rng(0).standard_normal(n).astype(np.float32)).cuda()
    new = lambda: dict(theta=torch.zeros(n, device="cuda"), grad=g.clone(), m=torch.zeros(n, device="cuda"),
                       v=torch.zeros(n, device="cuda"))
    want = new()
    L.AdamWGroup([want]).step(**hp)
    torch.cuda.synchronize()
    t = new()
    side = torch.cuda.Stream()
    group = L.AdamWGroup([t])
    tables, size = group._tables.data_ptr(), group._tables.numel()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(int(4e8))  # ~0.2 s: the step waits behind it
    group.step(**hp, stream=side)
    del group
    # nothing is written to what is handed out: the step may read it
    taken = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(64)]
    busy = not side.query()
    assert busy and tables not in [x.data_ptr() for x in taken]
    side.synchronize()
    for k in want:
        assert torch.equal(t[k], want[k]), k
