"""CPU model of the tensor-core scan's copies and products, and of its way out when a wait gives up.

One CTA walks over chunks.  Its loading thread starts copies of B, C and X into
shared memory, its issuing thread products that read them; each signals a
barrier of its own, one phase a chunk.  Copies and products complete in any
order and as late as they like.  A wait that gives up makes its thread go on
without waiting.  Whatever happens, no barrier may get an arrival for a phase
while the one before is open (its accounting breaks, and copies land over one
another), and nothing may be on its way when the CTA ends and its memory goes
to the next one.

The kernel's way out (vote at the chunk's end, leave, wait for everything that
was started) must pass; going on to the last chunk and waiting for the last
products only is the negative control that the model has to catch.
"""
import random

import pytest

B, C, X, G, READ, Y, S = range(7)      # the barriers: three copies; products that signal G, C read, Y and S


class Broken(Exception):
    pass


class Cta:
    def __init__(self, rng, give_up):
        self.rng, self.give_up = rng, give_up
        self.started, self.done = [0] * 7, [0] * 7
        self.ok = {"load": True, "issue": True, "rest": True}

    def start(self, *bars):
        for b in bars:
            if self.started[b] != self.done[b]:
                raise Broken("barrier %d gets an arrival in an open phase" % b)
            self.started[b] += 1
            if self.rng.random() < 0.3:
                self.done[b] += 1

    def wait(self, who, bar, k):
        """For phase k; a thread that gave up waits no more."""
        if not self.ok[who] or self.done[bar] > k:
            return
        assert self.started[bar] > k, "a wait for what nobody started"
        if self.rng.random() < self.give_up:
            self.ok[who] = False
        else:
            self.done[bar] = k + 1

    def wait_all(self, bar, k):
        for who in self.ok:
            self.wait(who, bar, k)

    def drain(self, bar, k):
        assert self.started[bar] > k, "a wait for what nobody started: it would last to its limit"
        self.done[bar] = k + 1


def run(chunks, ragged, state, seed, give_up, leave):
    """`ragged`: chunks with rows to clear; `state`: the launch that forms states only; `leave`: the kernel's way out."""
    cta = Cta(random.Random(seed), give_up)
    cta.start(X, B)
    if not state:
        cta.start(C)
    k = 0
    while k < chunks:
        more = k + 1 < chunks
        if k in ragged:
            cta.wait_all(B, k)
            cta.wait_all(X, k)
        if not state:
            cta.wait("issue", B, k)
            cta.wait("issue", C, k)
            cta.start(G, READ)
            cta.wait_all(X, k)
            cta.wait_all(G, k)
            cta.start(Y)
            cta.wait_all(READ, k)
        else:
            cta.wait_all(X, k)
            cta.wait_all(B, k)
        cta.start(S)
        if not state:
            cta.wait_all(Y, k)
        cta.wait_all(S, k)
        ahead = False
        if leave and more:
            cta.wait("load", B, k)
            if not state:
                cta.wait("load", C, k)
            ahead = cta.ok["load"]
        if more and (ahead or not leave):
            cta.start(*((B,) if state else (B, C)))
        if leave and not all(cta.ok.values()):
            for b in (S,) if state else (G, READ, Y, S):
                cta.drain(b, k)
            cta.drain(X, k)
            for b in (B,) if state else (B, C):
                cta.drain(b, k + ahead)
            break
        if more:
            cta.start(X)
        k += 1
    if not leave and not all(cta.ok.values()):
        for b in (S,) if state else (S, Y):
            cta.drain(b, chunks - 1)
    if cta.started != cta.done:
        raise Broken("something is on its way as the CTA ends")
    return k


CASES = [(1, (0,), False), (1, (), True), (4, (3,), False), (4, (3,), True), (6, (1, 5), False), (6, (1, 5), True)]


@pytest.mark.parametrize("chunks,ragged,state", CASES)
def test_a_wait_that_gives_up_leaves_nothing_behind(chunks, ragged, state):
    ends = {run(chunks, ragged, state, seed, 0.1, True) for seed in range(400)}
    assert len(ends) > 1 or chunks == 1           # some runs left early, some did not


@pytest.mark.parametrize("chunks,ragged,state", CASES)
def test_without_a_wait_that_gives_up_every_chunk_runs(chunks, ragged, state):
    assert {run(chunks, ragged, state, seed, 0.0, True) for seed in range(100)} == {chunks}
    assert {run(chunks, ragged, state, seed, 0.0, False) for seed in range(100)} == {chunks}


@pytest.mark.parametrize("chunks,ragged,state", CASES)
def test_going_on_after_a_wait_gave_up_is_caught(chunks, ragged, state):
    caught = 0
    for seed in range(400):
        try:
            run(chunks, ragged, state, seed, 0.4, False)
        except Broken:
            caught += 1
    assert caught >= 20
