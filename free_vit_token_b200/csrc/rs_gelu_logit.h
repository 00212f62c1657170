// Generated by gen_gelu_logit.py. GELU(z) = z / (1 + 2^(-z Q(min(z^2, T)))), Q of
// degree 3; max |error| 1.44e-05 in float32.
#pragma once
#define RS_GELU_LOGIT_T 25.0f
#define RS_GELU_LOGIT_Q0 2.301548633e+00f
#define RS_GELU_LOGIT_Q1 1.061382109e-01f
#define RS_GELU_LOGIT_Q2 -7.935004036e-04f
#define RS_GELU_LOGIT_Q3 -1.939556816e-05f
