// Generated by gen_exp2_poly.py: minimax (relative error) quintic for 2^f,
// f in [-1/2, 1/2], Remez exchange in float64; max relative error 7.494e-08.
#pragma once
#define CSA_EXP2_Q0 1.0000001f
#define CSA_EXP2_Q1 0.69314694f
#define CSA_EXP2_Q2 0.2402212f
#define CSA_EXP2_Q3 0.05550713f
#define CSA_EXP2_Q4 0.009675541f
#define CSA_EXP2_Q5 0.0013276472f
