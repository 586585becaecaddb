"""Entry points called by several host threads at once, each with its own
stream and workspace: the same results as one after the other, and no refusal."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


def _at_once(calls, repeats):
    """Each call in a host thread of its own, `repeats` times, all started together; raises what one of them raised."""
    start, errors = threading.Barrier(len(calls)), []

    def loop(call):
        start.wait()
        try:
            for _ in range(repeats):
                call()
        except Exception as e:
            errors.append(e)

    threads = [threading.Thread(target=loop, args=(call,)) for call in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    if errors:
        raise errors[0]


@pytest.mark.parametrize("accumulate", [False, True])
def test_embed_grad_of_different_sizes(accumulate):
    """Sizes of the sorted path whose shared memory differs: owners of 1,027 table rows and of 7. Sums of whole numbers
    are exact, so each call gives the definition's values."""
    from speculative_decoding_semi_b200 import binding as b
    calls, checks = [], []
    for n, V, r in [(20000, 151936, 8)] * 2 + [(6500, 1000, 8)] * 6:
        gen = torch.Generator(device="cuda").manual_seed(n)
        dout = torch.randint(-4, 5, (n, r), device="cuda", generator=gen).float()
        tokens = torch.randint(0, V, (n,), dtype=torch.int32, device="cuda", generator=gen)
        ws = torch.zeros(b.dspark_embed_grad_workspace_bytes(n, V, r), dtype=torch.uint8, device="cuda")
        dtable, stream = torch.zeros(V, r, device="cuda"), torch.cuda.Stream()
        scale = 0.0 if accumulate else 0.5            # what is added any number of times stays what it was
        if accumulate:
            dtable.fill_(3.0)
            want = dtable.clone()
        else:
            want = torch.zeros(V, r, device="cuda").index_add_(0, tokens, dout, alpha=0.5)
        calls.append(lambda a=(dout, tokens, scale, dtable, ws), s=stream:
                     b.dspark_embed_grad(*a, accumulate=accumulate, stream=s))
        checks.append((dtable, want, ws))
    torch.cuda.synchronize()
    _at_once(calls, 2000)
    for got, want, ws in checks:
        assert b.dspark_read_device_error(ws)[0] == 0
        assert torch.equal(got, want)


@pytest.mark.parametrize("sizes", [((512, 32), (64, 32)), ((200, 8), (3, 5))])
def test_schedule_of_different_sizes(sizes):
    """Both kernels (2,048 items and more, and fewer), each with two sizes of shared memory."""
    from speculative_decoding_semi_b200 import binding as b
    calls, checks = [], []
    for B, K in sizes * 3:
        gen = torch.Generator(device="cuda").manual_seed(B)
        conf, temps = torch.randn(B, K, device="cuda", generator=gen), torch.ones(K, device="cuda")
        profile = 1.0 + 0.01 * torch.arange(B * (K + 1) + 1, dtype=torch.float32, device="cuda")
        i32 = torch.int32
        outs = (torch.empty(B, dtype=i32, device="cuda"), torch.empty(B, K, device="cuda"),
                torch.empty(B, dtype=torch.int64, device="cuda"), torch.empty(1, dtype=i32, device="cuda"))
        ws = torch.zeros(b.dspark_workspace_bytes(B, K, 8, 1), dtype=torch.uint8, device="cuda")
        stream = torch.cuda.Stream()
        b.dspark_schedule(conf, temps, profile, *outs, ws)
        torch.cuda.synchronize()
        want = [o.clone() for o in outs]
        for o in outs:
            o.zero_()
        calls.append(lambda a=(conf, temps, profile, *outs, ws), s=stream: b.dspark_schedule(*a, s))
        checks.append((outs, want, ws))
    torch.cuda.synchronize()
    _at_once(calls, 2000)
    for outs, want, ws in checks:
        assert b.dspark_read_device_error(ws)[0] == 0
        for got, w in zip(outs, want):
            assert torch.equal(got, w)
