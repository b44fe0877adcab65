"""colibri_int_check and colibri_sync_status after device waits that ran out (colibri_moe_decode, int8
products).  A wait that nothing ever completes gives up after a short limit; nothing faults or hangs."""
import threading

import pytest
import torch

import sparse_expert_ffn_router_b200 as colibri
from tests import test_int_products as P
from tests.test_gpu_decode import BF16, F32, Case

TIMEOUT, INVALID = -6, -1


def _timed_out(stream=None):
    with pytest.raises(colibri.ColibriError) as ei:
        colibri.colibri_int_check(stream)
    assert ei.value.status == TIMEOUT and "gave up" in colibri.colibri_last_error()


@pytest.mark.parametrize("bad", [0, -5, 1000001])
def test_selftest_refuses(bad):
    with pytest.raises(colibri.ColibriError) as ei:
        colibri.colibri_int_selftest_wait_timeout(bad)
    assert ei.value.status == INVALID and colibri.colibri_last_error()


@pytest.mark.gpu
def test_a_wait_that_ran_out_is_reported_once():
    prob = P._problem(40, 300, 512, 4)
    good = P._run_gemm(*prob, F32)
    colibri.colibri_int_check()
    streams = [None, torch.cuda.Stream(), torch.cuda.Stream()]
    for raised in streams:
        for asked in streams:
            colibri.colibri_int_selftest_wait_timeout(500, raised)
            if asked is not raised:  # a check waits for its own stream only
                torch.cuda.synchronize()
            _timed_out(asked)
            for st in streams:
                colibri.colibri_int_check(st)
    colibri.colibri_int_selftest_wait_timeout(500, streams[1])
    assert torch.equal(P._run_gemm(*prob, F32, stream=streams[1]), good)  # products run as before
    _timed_out(streams[1])
    colibri.colibri_int_check(streams[1])


@pytest.mark.gpu
def test_a_context_and_the_products_have_words_of_their_own():
    c = Case(2, 64, 64, 2, 1)
    colibri.colibri_int_selftest_wait_timeout(200)
    c.layer.sync_status()
    _timed_out()
    colibri.colibri_selftest_wait_timeout(c.layer.ctx, 200)
    colibri.colibri_int_check()
    with pytest.raises(colibri.ColibriError) as ei:
        c.layer.sync_status()
    assert ei.value.status == TIMEOUT


@pytest.mark.gpu
def test_checks_from_several_threads_report_every_round():
    # four threads, each with a stream: in a round one wait runs out and all check; exactly one is told
    n, rounds = 4, 40
    streams = [torch.cuda.Stream() for _ in range(n)]
    told = [[0] * rounds for _ in range(n)]
    gate, errors = threading.Barrier(n), []

    def work(i):
        try:
            for r in range(rounds):
                gate.wait(60)
                if i == 0:
                    colibri.colibri_int_selftest_wait_timeout(50, streams[r % n])
                    streams[r % n].synchronize()
                gate.wait(60)
                try:
                    colibri.colibri_int_check(streams[i])
                except colibri.ColibriError as e:
                    assert e.status == TIMEOUT
                    told[i][r] = 1
        except BaseException as e:  # noqa: BLE001
            errors.append(e)
            gate.abort()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(n)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    assert [sum(t[r] for t in told) for r in range(rounds)] == [1] * rounds


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("d", [128, 2048])  # with and without the third grid barrier of the launch
def test_decode_after_a_wait_that_ran_out(d, dt):
    # the launch's grid-barrier counters have advanced before the error, and the status call resets them
    c = Case(5, d, 192, 6, 2, 64, dt)
    first = c.decode()
    c.check(first)
    for _ in range(3):
        colibri.colibri_selftest_wait_timeout(c.layer.ctx, 300)
        with pytest.raises(colibri.ColibriError) as ei:
            c.layer.sync_status()
        assert ei.value.status == TIMEOUT
        c.layer.sync_status()
        for _ in range(2):
            y = c.decode()
            c.layer.sync_status()
            assert torch.equal(y, first)
