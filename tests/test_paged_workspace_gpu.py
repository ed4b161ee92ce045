"""Device memory that the binding keeps for the paged calls: bounded a
thread, released with the thread."""
import threading

import pytest

from test_paged_gpu import Batch, S, forward  # noqa: F401

pytestmark = pytest.mark.gpu


def held(cuda):
    import gc
    gc.collect()
    cuda.cuda.synchronize()
    return cuda.cuda.memory_allocated()


def one_workspace(S):
    p = S.SdpaPagedParams()
    p.num_seqs = p.num_tokens = p.num_q_heads = p.num_kv_heads = p.page_size = 1
    p.head_dim, p.scale = 64, 1.0
    return S.sdpa_paged_workspace_size(p)


def in_thread(work):
    errors = []

    def run():
        try:
            work()
        except BaseException as e:  # noqa: BLE001
            errors.append(e)

    th = threading.Thread(target=run)
    th.start()
    th.join()
    if errors:
        raise errors[0]


def test_a_threads_workspaces_go_with_it(cuda, S):
    t = Batch(cuda, [1, 9], [300, 70], 8, 2, 64, "bf16", 16)
    ref = forward(S, t)
    before = held(cuda)
    alive = [threading.Event() for _ in range(6)]
    for e in alive:  # threads one after another (their identifiers may repeat) and at once
        in_thread(lambda: forward(S, t))
    done = threading.Event()

    def stay(e):
        forward(S, t)
        e.set()
        done.wait(60)

    th = [threading.Thread(target=stay, args=(e,)) for e in alive]
    [x.start() for x in th]
    [e.wait(60) for e in alive]
    done.set()
    [x.join() for x in th]
    assert held(cuda) - before < one_workspace(S)
    o, lse = forward(S, t)
    assert cuda.equal(o, ref[0]) and cuda.equal(lse, ref[1])


def test_many_streams_of_one_thread(cuda, S):
    t = Batch(cuda, [1, 300], [900, 700], 8, 2, 64, "bf16", 16)
    ref = forward(S, t)
    cuda.cuda.synchronize()
    size = one_workspace(S)

    def work():
        before = held(cuda)
        streams = [cuda.cuda.Stream() for _ in range(12)]
        outs = []
        for _ in range(3):  # the streams in turn: workspaces are dropped while their calls run
            for s in streams:
                with cuda.cuda.stream(s):
                    outs.append(forward(S, t))
        cuda.cuda.synchronize()
        for o, lse in outs:
            assert cuda.equal(o, ref[0]) and cuda.equal(lse, ref[1])
        del outs, o, lse
        assert held(cuda) - before <= 5 * size

    in_thread(work)
