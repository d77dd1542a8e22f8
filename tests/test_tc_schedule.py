"""The barrier schedule of the block-scaled product on tcgen05, on a host model (no GPU).

One thread copies block i into stage i mod S, issuing thread i mod 2 multiplies it into buffer i mod B, one warp
brings the block's scales and others read the buffer back. Copies and products complete in any order that the
hardware leaves open; the barriers count arrivals by phases, and a wait by parity sees whether the open phase has
the other parity. The model checks that a product never reads a stage that does not hold its block, that no copy
starts over a stage still being read, and that everything ends.
"""
import os
import random
import shutil
import subprocess

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "mixture_experts_grouped_gb300", "csrc")
WIDTHS = [256, 128, 64]  # of the tiles


class Barrier:
    def __init__(self, count):
        self.count, self.pending, self.phase = count, count, 0

    def arrive(self):
        self.pending -= 1
        if self.pending == 0:
            self.phase, self.pending = self.phase + 1, self.count

    def done(self, parity):
        """mbarrier.try_wait.parity: the phase before the open one has this parity."""
        return (self.phase - 1) % 2 == parity


class Fault(Exception):
    pass


def run(stages, bufs, blocks, issuers, rng):
    full = [Barrier(2) for _ in range(stages)]     # the copying thread's arrival, and its bytes
    empty = [Barrier(1) for _ in range(stages)]
    tfull = [Barrier(2) for _ in range(bufs)]      # the products, and the scales
    tempty = [Barrier(1) for _ in range(bufs)]
    holds = [None] * stages                        # the block whose bytes a stage holds
    reading = [0] * stages                         # products in flight that read it
    copies, products = [], [[] for _ in range(issuers)]

    def copier():
        for i in range(blocks):
            s = i % stages
            while not empty[s].done((i // stages + 1) % 2):
                yield False
            if reading[s]:
                raise Fault(f"copy of block {i} over a stage that is being read")
            holds[s] = None
            full[s].arrive()
            copies.append(i)
            yield True

    def issuer(w):
        for i in range(w, blocks, issuers):
            s, b = i % stages, i % bufs
            while not full[s].done(i // stages % 2):
                yield False
            while not tempty[b].done((i // bufs + 1) % 2):
                yield False
            if holds[s] != i:
                raise Fault(f"product of block {i} on a stage that holds {holds[s]}")
            reading[s] += 1
            products[w].append(i)
            yield True

    def scaler():
        for i in range(blocks):
            while not tempty[i % bufs].done((i // bufs + 1) % 2):
                yield False
            tfull[i % bufs].arrive()
            yield True

    def reader():
        for i in range(blocks):
            while not tfull[i % bufs].done(i // bufs % 2):
                yield False
            tempty[i % bufs].arrive()
            yield True

    def lander():  # copies land in any order
        while True:
            if copies:
                i = copies.pop(rng.randrange(len(copies)))
                holds[i % stages] = i
                full[i % stages].arrive()
            yield bool(copies)

    def finisher(w):  # a thread's products complete in its order
        while True:
            if products[w]:
                i = products[w].pop(0)
                reading[i % stages] -= 1
                tfull[i % bufs].arrive()
                empty[i % stages].arrive()
            yield bool(products[w])

    work = [copier(), scaler(), reader()] + [issuer(w) for w in range(issuers)]
    hardware = [lander()] + [finisher(w) for w in range(issuers)]
    weight = {id(g): rng.choice([1, 1, 4, 16]) for g in work + hardware}  # some run late, some early
    idle = 0
    while work:
        g = rng.choices(work + hardware, [weight[id(x)] for x in work + hardware])[0]
        try:
            moved = next(g)
        except StopIteration:
            work.remove(g)
            moved = True
        idle = 0 if moved else idle + 1
        if idle > 20000:
            raise Fault("nothing moves")


def faults(stages, bufs, issuers, tries=400, blocks=25):
    rng = random.Random(stages * 100 + bufs)
    bad = []
    for _ in range(tries):
        try:
            run(stages, bufs, blocks, issuers, rng)
        except Fault as f:
            bad.append(str(f))
    return bad


@pytest.fixture(scope="module")
def rings(tmp_path_factory):
    """(stages, buffers) of every tile width and the issuing threads, from the header that the kernel is built with."""
    d = tmp_path_factory.mktemp("ring")
    src = d / "ring.cpp"
    calls = "".join(f'std::printf("%d %d\\n", moe::tc_stages({bn}), moe::tc_buffers({bn}));\n'
                    for bn in WIDTHS)
    src.write_text('#include <cstdio>\n#include "tc_ring.cuh"\nint main() {\n'
                   'std::printf("%d\\n", moe::kTcIssuers);\n' + calls + "}\n")
    exe = d / "ring"
    subprocess.run([shutil.which("g++") or "g++", "-std=c++17", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    lines = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split("\n")
    return int(lines[0]), {f: tuple(map(int, l.split())) for f, l in zip(WIDTHS, lines[1:])}


@pytest.mark.parametrize("width", WIDTHS)
def test_no_product_reads_a_stage_that_has_not_arrived(rings, width):
    issuers, shape = rings
    bad = faults(*shape[width], issuers)
    assert not bad, f"{len(bad)} of 400 orders: {bad[0]}"


def test_the_model_sees_a_stage_shared_by_two_threads():
    assert any("product of block" in f for f in faults(5, 4, 2))
    assert not faults(5, 4, 1)
