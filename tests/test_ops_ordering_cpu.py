"""Orderings in the operators' kernels that no run shows: they are read from
the sources, since what breaks one depends on how far blocks drift apart."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "exact_bpe_tokenization_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name), encoding="utf-8") as f:
        return re.sub(r"//[^\n]*|^[ \t]*#[^\n]*", "", f.read(), flags=re.M)


def body_of(text, start):
    """The braces' content behind the first match of `start`."""
    i = text.index("{", re.search(start, text).end())
    depth, j = 0, i
    while True:
        depth += {"{": 1, "}": -1}.get(text[j], 0)
        j += 1
        if depth == 0:
            return text[i + 1:j - 1]


class Walk:
    """The ways through a body of statements, lambdas followed where they are
    called.  A way's state is whether a block may still have to read the sums
    that the blocks of its cluster told it; `broken` lists where some way tells
    new ones in that state."""
    TOKEN = re.compile(r"[A-Za-z_]\w*|[(){};=\[\]]")
    READS, TELLS, BARRIER = {"row_total"}, {"push_sums", "block_totals"}, {"sync_row"}

    def __init__(self, text):
        self.t = self.TOKEN.findall(text) + ["}"]
        self.i, self.lambdas, self.broken = 0, {}, []

    # -- statements
    def parens(self):
        """Events within one pair of parentheses."""
        out, depth = [], 0
        while True:
            t = self.t[self.i]
            depth += {"(": 1, ")": -1}.get(t, 0)
            self.event(t, out)
            self.i += 1
            if depth == 0:
                return out

    def event(self, t, out):
        if self.t[self.i + 1] == "(" and (t in self.READS | self.TELLS | self.BARRIER or t in self.lambdas):
            out.append(t)

    def block(self):
        out = []
        while self.t[self.i] != "}":
            out.append(self.statement())
        self.i += 1
        return ("all", out)

    def statement(self):
        t = self.t[self.i]
        if t == "{":
            self.i += 1
            return self.block()
        if t == "if":
            self.i += 1 + (self.t[self.i + 1] == "constexpr")
            events, yes, no = self.parens(), self.statement(), ("all", [])
            if self.t[self.i] == "else":
                self.i += 1
                no = self.statement()
            return ("if", events, yes, no)
        if t in ("for", "while"):
            self.i += 1
            endless = self.t[self.i:self.i + 4] == ["(", ";", ";", ")"]
            return ("loop", self.parens(), self.statement(), endless)
        if t == "auto" and self.t[self.i + 2:self.i + 4] == ["=", "["]:
            name = self.t[self.i + 1]
            while self.t[self.i] != "(":
                self.i += 1
            self.parens()
            self.i += 1
            self.lambdas[name] = self.block()
            self.i += 1
            return ("all", [])
        events, depth = [], 0
        while self.t[self.i] != ";" or depth:
            depth += {"(": 1, "{": 1, ")": -1, "}": -1}.get(self.t[self.i], 0)
            self.event(self.t[self.i], events)
            self.i += 1
        self.i += 1
        return ("return" if t == "return" else "do", events)

    # -- states: the sets behind a statement, and behind a return
    def do(self, events, states, at):
        for e in events:
            if e in self.lambdas:
                after, returned = self.run(self.lambdas[e], states, at + [e])
                states = after | returned
            elif e in self.READS:
                states = {True for _ in states}
            elif e in self.BARRIER:
                states = {False for _ in states}
            elif True in states:
                self.broken.append(" > ".join(at + [e]))
        return states

    def run(self, node, states, at=[]):
        kind, returned = node[0], set()
        if kind == "all":
            for n in node[1]:
                states, r = self.run(n, states, at)
                returned |= r
        elif kind == "if":
            states = self.do(node[1], states, at)
            (a, r1), (b, r2) = self.run(node[2], states, at), self.run(node[3], states, at)
            states, returned = a | b, r1 | r2
        elif kind == "loop":
            seen = set()
            while not states <= seen:
                seen |= states
                states, r = self.run(node[2], self.do(node[1], seen, at), at)
                returned |= r
            states = set() if node[3] else seen | states
        else:
            states = self.do(node[1], states, at)
            if kind == "return":
                states, returned = set(), states
        return states, returned


def walk(text):
    w = Walk(text)
    w.run(w.block(), {False})
    return w.broken


def test_the_walk_follows_ways():
    """What it finds and what it passes, on small bodies."""
    assert walk("push_sums(x); sync_row(); t = row_total(); sync_row(); push_sums(y);") == []
    assert walk("push_sums(x); sync_row(); t = row_total(); push_sums(y);") == ["push_sums"]
    assert walk("t = row_total(); if (a) sync_row(); push_sums(y);") == ["push_sums"]
    assert walk("t = row_total(); if (a) sync_row(); else { sync_row(); } push_sums(y);") == []
    assert walk("auto f = [&](int n) { if (n) return; push_sums(n); }; t = row_total(); f(1);") == ["f > push_sums"]
    assert walk("auto f = [&](int n) { sync_row(); }; t = row_total(); f(1); push_sums(2);") == []
    assert walk("for (;;) { push_sums(x); sync_row(); if (a) return; t = row_total(); }")
    assert walk("for (;;) { push_sums(x); sync_row(); t = row_total(); if (a) return; sync_row(); }") == []


def test_a_rows_sums_are_read_before_new_ones_are_told():
    """Blocks of a cluster write their sums into one another's shared memory: a
    cluster barrier stands between every reading of them and the next telling,
    on every way through the histograms."""
    text = source("tt_sample.cu")
    body = body_of(text, r"void sample_by_bins\(")
    assert len(re.findall(r"row_total\(", body)) >= 4 and "prefix_end" in body
    assert walk(body) == []
    assert walk(body_of(text, r"bool sample_by_list\(")) == []


def test_chained_kernels_take_only_the_callers_inputs_as_constant():
    """A kernel that is there before the one ahead of it ends may declare
    constant (const __restrict__) only what no kernel of the call writes."""
    inputs = {"ids", "table", "dout", "logits"}             # parameters that the calls' own inputs are given to
    chained = {}
    for name in ("tt_embed.cu", "tt_loss.cu", "tt_sample.cu"):
        text = source(name)
        for m in re.finditer(r"__global__[^;{]*?(k_\w+)\(([^{;]*)\)\s*\{", text):
            if "wait_for_last()" in body_of(text, re.escape(m[0][:-1])):
                chained[m[1]] = set(re.findall(r"const \w+ \*__restrict__ (\w+)", m[2]))
    assert {"k_sort_place", "k_sort_scan", "k_grad_sum", "k_grad_join", "k_sample_bins"} <= set(chained)
    assert not {k: v - inputs for k, v in chained.items() if v - inputs}
